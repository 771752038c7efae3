"""The native module's calls on arguments that PyTorch itself refuses, on the CPU: an exception has to
reach Python, not end the interpreter, and a HIP error that an entry point reports has to reach it too,
without a second call.  They run in a process of their own.  Fake tensors stand for GPU tensors: they
say they are on the GPU and hold no memory."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SETUP = """
import torch
import fp8_delayed_scaling_amd as F
from torch._subclasses.fake_tensor import FakeTensorMode

mode = FakeTensorMode()
with mode:
    bf = dict(dtype=torch.bfloat16, device="cuda")
    u8, f32, i32 = (dict(dtype=t, device="cuda") for t in (torch.uint8, torch.float32, torch.int32))
    x, w, s = torch.empty(4, 32, **bf), torch.empty(32, **bf), torch.empty(1, **f32)
    codes, experts, weights = torch.empty(3, 64, 32, **u8), torch.empty(4, 2, **i32), torch.empty(4, 2, **f32)
    src, off, ys = torch.empty(64, **i32), torch.empty(4, **i32), torch.empty(64, 32, **bf)
    many = torch.empty(3, 4, 32, **bf), torch.empty(3, 64, 32, **bf), torch.empty(3, 4, 2, **i32), torch.empty(3, 64, 32, **u8)
"""


def _run(code):
    r = subprocess.run([sys.executable, "-W", "ignore", "-c", SETUP + code], cwd=ROOT, capture_output=True, text=True, timeout=120,
                       env=dict(os.environ, HIP_VISIBLE_DEVICES="-1"))
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout.strip().splitlines()


CALLS = {
    "norm_fwd": "F.fp8_norm_residual_fwd(x, w, None, None, x, 1.0, x, None, w, None, None, x, stream={s})",
    "norm_bwd": "F.fp8_norm_residual_bwd(x, x, None, None, None, None, 1.0, x, None, w, weights, None, x, None, None, None, None, None, s, "
                "stream={s})",
    "moe_plan": "F.fp8_moe_plan(experts, 3, 16, off, src, experts, stream={s})",
    "moe_sort_cast": "F.fp8_moe_sort_cast(x, src, 2, None, s, 0, codes[0], stream={s})",
    "moe_sort_codes": "F.fp8_moe_sort_codes(codes[0, :4], src, 2, codes[0], stream={s})",
    "moe_combine": "F.fp8_moe_combine(ys, experts, weights, x, stream={s})",
    "moe_weight_grad": "F.fp8_moe_weight_grad(x, ys, experts, weights, stream={s})",
    "grouped_gemm": "F.fp8_grouped_gemm(codes[0], 0, s, codes[:, :32], 0, s, off, ys, stream={s})",
    "grouped_wgrad": "F.fp8_grouped_wgrad(codes[0], 0, s, codes[1], 0, s, off[:2], torch.empty(1, 64, 64, **bf), stream={s})",
}


TRY = """
def attempt(name, fn):
    try:
        with mode:
            fn()
        print(name, "returned", flush=True)
    except Exception as e:
        print(name, type(e).__name__, str(e).splitlines()[0], flush=True)
"""


def test_no_current_stream():
    """Without a GPU there is no current stream: asking for it raises."""
    out = _run(TRY + "".join(f"attempt({name!r}, lambda: {call.format(s=None)})\n" for name, call in CALLS.items()))
    assert len(out) == len(CALLS)
    for line, name in zip(out, CALLS):
        assert line.startswith(name + " ") and any(k in line for k in ("GPU", "HIP", "CUDA")), line


def test_tensors_without_memory():
    """Inside vmap a tensor has no storage of its own: its pointer cannot be taken."""
    batched = {"norm_fwd": 0, "norm_bwd": 0, "moe_sort_cast": 0, "moe_combine": 1, "moe_weight_grad": 1, "moe_plan": 2,
               "moe_sort_codes": 3, "grouped_gemm": 3, "grouped_wgrad": 3}
    code = TRY
    for name, call in CALLS.items():
        var = ("x", "ys", "experts", "codes0")[batched[name]]
        call = call.format(s=0)
        if var == "codes0":
            call = call.replace("codes[0, :4]", "codes0[:4]").replace("codes[0]", "codes0")
        code += f"""
def f({var}):
    {call}
    return {var}
attempt({name!r}, lambda: torch.vmap(f)(many[{batched[name]}]))
"""
    out = _run(code)
    assert len(out) == len(CALLS)
    for line, name in zip(out, CALLS):
        assert line.startswith(name + " RuntimeError") and ("data pointer" in line or "storage" in line), line


def test_streams_that_are_no_handle():
    """No error of the conversion is left behind: what is raised is the binding's own."""
    streams = ("1 << 70", "-(1 << 70)", "object()", "type('S', (), dict(cuda_stream='x'))()")
    out = _run(TRY + "".join(f"attempt('stream', lambda: {CALLS['norm_fwd'].format(s=s)})\n" for s in streams))
    assert len(out) == len(streams)
    for line in out:
        assert line.split()[1] in ("Fp8dsError", "AttributeError", "TypeError", "ValueError", "ArgumentError"), line


ENTRIES = {name: ("fp8_norm_residual_" + name[5:] if name.startswith("norm") else "fp8_" + name) for name in CALLS}
# Entry points that count their calls and report what they are told to; loaded for all, so that they take the library's place.
STUB = "int status, calls;\n" + "".join(f"int {e}(void) {{ ++calls; return status; }}\n" for e in ENTRIES.values())


def _stub(tmp_path):
    (tmp_path / "stub.c").write_text(STUB)
    out = str(tmp_path / "stub.so")
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", out, str(tmp_path / "stub.c")], check=True)
    return f"""
import ctypes
stub = ctypes.CDLL({out!r}, ctypes.RTLD_GLOBAL)
status, calls = ctypes.c_int.in_dll(stub, "status"), ctypes.c_int.in_dll(stub, "calls")
"""


def test_a_hip_error_is_raised_and_the_call_is_not_made_again(tmp_path):
    """An entry point that reports a HIP error may have launched: a second call would run it twice, and with
    x in resid's buffer the first norm would be added twice."""
    code = _stub(tmp_path) + TRY + "F._invoke = lambda *a: print('again', a[0], flush=True)\nstatus.value = -6\n"
    code += "".join(f"attempt({name!r}, lambda: {call.format(s=0)})\n" for name, call in CALLS.items()) + "print(calls.value)\n"
    out = _run(code)
    assert out[-1] == str(len(CALLS)) and len(out) == len(CALLS) + 1, out
    for line, name in zip(out, CALLS):
        assert line.startswith(f"{name} Fp8dsError FP8DS_ERR_HIP"), line


def test_a_refusal_is_left_to_the_bindings_checks(tmp_path):
    code = _stub(tmp_path) + TRY + "F._invoke = lambda *a: print('again', a[0], flush=True)\n"
    refusals = (-1, -2, -3, -4, -5, -7)
    for value in (*refusals, 0):
        code += f"status.value = {value}\nattempt('norm', lambda: {CALLS['norm_fwd'].format(s=0)})\n"
    out = _run(code + "print(calls.value)\n")
    assert out == ["again fp8_norm_residual_fwd", "norm returned"] * len(refusals) + ["norm returned", str(len(refusals) + 1)], out


def test_other_threads_run_during_a_call(tmp_path):
    """A launch may wait for the GPU: the entry point here waits, at most two seconds, for another thread."""
    (tmp_path / "wait.c").write_text("""
#include <unistd.h>
volatile int flag, seen;
int fp8_moe_combine(void) {
    for (int i = 0; i < 2000 && !flag; ++i) usleep(1000);
    seen = flag;
    return 0;
}
""")
    lib = str(tmp_path / "wait.so")
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", lib, str(tmp_path / "wait.c")], check=True)
    out = _run(f"""
import ctypes, threading
stub = ctypes.CDLL({lib!r}, ctypes.RTLD_GLOBAL)
flag, seen = ctypes.c_int.in_dll(stub, "flag"), ctypes.c_int.in_dll(stub, "seen")
other = threading.Timer(0.05, lambda: setattr(flag, "value", 1))
other.start()
with mode:
    {CALLS["moe_combine"].format(s=0)}
print(seen.value)
other.join()
""")
    assert out == ["1"]
