"""Wait states of the built library's LDS DMA, which the hardware does not interlock and which the compiler does not
look for inside inline assembly: one behind the write of M0, which holds the LDS address, and five behind a vector
instruction's write of a scalar register that the DMA reads."""
import os
import re
import struct
import subprocess

import dispatch_fp8_grouped_amd as mm

LLVM = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin")
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"
WRITES_M0 = re.compile(r"[sv]_\w+\s+m0\b")
LDS_DMA = re.compile(r"(global_load_lds_|buffer_load_lds_|buffer_load_\w+ .*\blds\b)")
SGPR = re.compile(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b")


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


def scalars(text):
    return {i for m in SGPR.finditer(text)
            for i in (range(int(m[1]), int(m[2]) + 1) if m[1] else [int(m[3])])}


def young_operand(before, dma):
    """Whether one of the last instructions (latest first) is a vector instruction that writes a scalar register of
    the DMA fewer than five wait states ahead of it."""
    states, reads = 0, scalars(dma)
    for line in before:
        name, _, rest = line.partition(" ")
        if name.startswith("v_") and scalars(rest.split(",")[0]) & reads:
            return True
        states += int(rest, 0) + 1 if name == "s_nop" else 1
        if states >= 5:
            break
    return False


def test_the_scan_sees_what_it_looks_for():
    dma = "buffer_load_dwordx4 v2, s[4:7], 0 offen lds"
    assert LDS_DMA.match(dma) and LDS_DMA.match("global_load_lds_dwordx4 v1, s[2:3]")
    assert not LDS_DMA.match("buffer_load_dwordx4 v[2:5], v2, s[4:7], 0 offen")
    assert WRITES_M0.match("s_mov_b32 m0, s34") and not WRITES_M0.match("s_mov_b32 s1, m0")
    assert young_operand(["s_nop 0", "s_mov_b32 m0, s9", "v_readfirstlane_b32 s5, v1"], dma)
    assert not young_operand(["s_nop 2", "s_mov_b32 m0, s9", "s_nop 0", "v_readfirstlane_b32 s5, v1"], dma)
    assert not young_operand(["s_nop 0", "s_mov_b32 m0, s9", "v_readfirstlane_b32 s8, v1"], dma)


def test_wait_states_ahead_of_the_dma(tmp_path):
    dma = 0
    for i, code in enumerate(device_code(mm.LIB_PATH, str(tmp_path))):
        obj = tmp_path / f"{i}.co"
        obj.write_bytes(code)
        with subprocess.Popen([os.path.join(LLVM, "llvm-objdump"), "-d", "--mcpu=gfx950", "--no-show-raw-insn", str(obj)],
                              stdout=subprocess.PIPE, text=True) as run:
            before, early = [], []
            for line in run.stdout:
                line = line.split("//")[0].strip()
                if not line:
                    continue
                if LDS_DMA.match(line):
                    dma += 1
                    if (before and WRITES_M0.match(before[0])) or young_operand(before, line):
                        early.append(before[::-1] + [line])
                before = [line] + before[:4]
        assert run.returncode == 0
        assert not early, (i, len(early), early[:2])
    assert dma > 1000          # the products' loops are there and were read
