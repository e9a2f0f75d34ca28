"""Child process of test_block_host_sanitizers.py (not a test module itself).

Drives every entry point of include/dg_block.h in the sanitizer-built library
through its argument checks and launch preparation, one and two arguments away
from a valid call, with fake device addresses that the host code never
dereferences.  Without a GPU a call that passes its checks fails at the launch.
No torch import: only ctypes touches the library.

usage: python block_host_sanitizer_driver.py LIB HEADER
"""

import ctypes
import re
import sys

FAKE = 1 << 24
TYPES = {"int": ctypes.c_int, "int64_t": ctypes.c_int64, "size_t": ctypes.c_size_t, "float": ctypes.c_float}
VALID = dict(
    tokens=64, cols=512, ld_y=512, ld_h=512, ld_r=512, ld_x=512, ld_sf=64, ld_dx=512, ld_dr=512, ld_dy=512, ld_dh=512, kind=0, post=1,
    gate_kind=1, res_scale=1.0, eps=1e-6, experts=256, topk=8, num_seqs=4, ld_logits=256, ld_add=256, ld_dlogits=256, score=1, coef=1.0,
    m=64, n=512, k=512, lda=512, ldb=512, ldd=512, ld_sfa=64, ld_res=512, ld_pre=512, ld_dsf=256, act=2, rows=256, ld_dd=512, ld_dsft=512,
    workspace_bytes=1 << 40)
TRIES = {"int": [-2**31, -1, 0, 1, 2, 3, 7, 127, 128, 129, 1 << 16, 1 << 20, 2**31 - 128, 2**31 - 1],
         "int64_t": [-2**63, -1, 0, 1, 4, 8, 1 << 20, 1 << 40, 1 << 62, 2**63 - 16, 2**63 - 1],
         "size_t": [0, 1, 2**64 - 1], "float": [0.0, 1e-45, 1e30, float("inf"), float("nan")]}


def declarations(header):
    text = re.sub(r"/\*.*?\*/", "", open(header).read(), flags=re.S)
    out = {}
    for ret, name, args in re.findall(r"(int|size_t)\s+(dg_\w+)\s*\(([^)]*)\)\s*;", text):
        params = []
        for arg in " ".join(args.split()).split(","):
            ctype, pname = arg.strip().rsplit(" ", 1)
            params.append((ctype + "*" * pname.startswith("*"), pname.lstrip("*")))
        out[name] = (ret, params)
    return out


def main():
    lib, decls, calls = ctypes.CDLL(sys.argv[1]), declarations(sys.argv[2]), 0
    lib.dg_get_last_error_string.restype = ctypes.c_char_p
    for name, (ret, params) in decls.items():
        fn = getattr(lib, name)
        fn.restype = TYPES[ret]
        fn.argtypes = [ctypes.c_void_p if "*" in t else TYPES[t] for t, _ in params]
        base = [(None if p == "stream" else FAKE) if "*" in t else VALID[p] for t, p in params]
        st = fn(*base)
        calls += 1
        assert ret == "size_t" or st == -5, f"{name}: {st} {lib.dg_get_last_error_string()}"
        for i, (ctype, pname) in enumerate(params):
            for v in ([0, FAKE + 1, FAKE + 4] if pname != "stream" else []) if "*" in ctype else TRIES[ctype]:
                for also in range(len(params)):  # and with one more argument at an extreme
                    args = list(base)
                    args[i] = v
                    t2, p2 = params[also]
                    if also != i and t2 in ("int", "int64_t"):
                        args[also] = TRIES[t2][(calls * 7) % len(TRIES[t2])]
                    st = fn(*args)
                    calls += 1
                    if ret == "int":
                        assert st in (0, -1, -2, -3, -4, -5), f"{name} {pname}={v}: {st}"
                        assert st == 0 or lib.dg_get_last_error_string(), f"{name} {pname}={v}: no message"
    print(f"block host-sanitizer driver ok calls={calls} entries={len(decls)}", flush=True)


if __name__ == "__main__":
    main()
