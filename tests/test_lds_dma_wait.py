"""Every LDS DMA of the built library comes at least one wait state behind the write of M0, which holds its LDS
address: the hardware does not interlock the two, and the compiler does not look into inline assembly."""
import os
import re
import struct
import subprocess

import dispatch_fp8_grouped_amd as mm

LLVM = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin")
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"
WRITES_M0 = re.compile(r"\s*[sv]_\w+\s+m0\b")
LDS_DMA = re.compile(r"\s*(global_load_lds_|buffer_load_lds_|buffer_load_\w+ .*\blds\b)")


def device_code(path, tmp):
    """The gfx950 code objects of a library: the .hip_fatbin section holds one bundle per source."""
    section = os.path.join(tmp, "fatbin")
    subprocess.run([os.path.join(LLVM, "llvm-objcopy"), "--dump-section", f".hip_fatbin={section}", path,
                    os.path.join(tmp, "copy")], check=True)
    data = open(section, "rb").read()
    for at in (m.start() for m in re.finditer(re.escape(MAGIC), data)):
        p = at + len(MAGIC) + 8
        for _ in range(struct.unpack_from("<Q", data, at + len(MAGIC))[0]):
            offset, size, n = struct.unpack_from("<QQQ", data, p)
            name = data[p + 24:p + 24 + n].decode()
            p += 24 + n
            if "gfx950" in name and size:
                yield data[at + offset:at + offset + size]


def test_a_wait_state_between_m0_and_the_dma(tmp_path):
    dma = 0
    for i, code in enumerate(device_code(mm.LIB_PATH, str(tmp_path))):
        obj = tmp_path / f"{i}.co"
        obj.write_bytes(code)
        with subprocess.Popen([os.path.join(LLVM, "llvm-objdump"), "-d", "--mcpu=gfx950", "--no-show-raw-insn", str(obj)],
                              stdout=subprocess.PIPE, text=True) as run:
            before, early = "", []
            for line in run.stdout:
                if LDS_DMA.match(line):
                    dma += 1
                    if WRITES_M0.match(before):
                        early.append(before.strip() + " ; " + line.strip())
                if line.strip():
                    before = line
        assert run.returncode == 0
        assert not early, (i, len(early), early[:3])
    assert dma > 1000          # the products' loops are there and were read
