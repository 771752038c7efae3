"""As test_call_errors.py, for the calls of attention and of the router: what PyTorch refuses and what an entry point
reports reach Python, once."""
import subprocess

from test_call_errors import TRY, _run

MORE = """
with mode:
    q, out, k, v = (torch.empty(6, 2, 16, **bf) for _ in range(4))
    lse, wsp = torch.empty(2, 6, **f32), torch.empty(4096, **u8)
    logits, ex, we, le = torch.empty(6, 8, **f32), torch.empty(6, 2, **i32), torch.empty(6, 2, **f32), torch.empty(6, **f32)
    counts, sums, loss = torch.empty(9, **i32), torch.empty(8, **f32), torch.empty(1, **f32)
    many = torch.empty(3, 6, 2, 16, **bf), torch.empty(3, 6, 8, **f32)
"""
CALLS = {
    "attention_fwd": "F.fp8_attention_fwd(q, k, v, out, lse, workspace=wsp, stream={s})",
    "attention_bwd": "F.fp8_attention_bwd(q, q, k, v, out, lse, out, out, out, wsp, stream={s})",
    "moe_route": "F.fp8_moe_route(logits, ex, we, le, counts, sums, loss, stream={s})",
    "moe_route_bwd": "F.fp8_moe_route_bwd(logits, ex, we, le, counts, we, loss, logits, stream={s})",
}


def test_no_current_stream():
    out = _run(MORE + TRY + "".join(f"attempt({n!r}, lambda: {c.format(s=None)})\n" for n, c in CALLS.items()))
    assert len(out) == len(CALLS)
    for line, name in zip(out, CALLS):
        assert line.startswith(name + " ") and any(k in line for k in ("GPU", "HIP", "CUDA")), line


def test_tensors_without_memory():
    code = MORE + TRY
    for name, call in CALLS.items():
        var, i = ("q", 0) if name.startswith("att") else ("logits", 1)
        code += f"""
def f({var}):
    {call.format(s=0)}
    return {var}
attempt({name!r}, lambda: torch.vmap(f)(many[{i}]))
"""
    out = _run(code)
    assert len(out) == len(CALLS)
    for line, name in zip(out, CALLS):
        assert line.startswith(name + " RuntimeError") and ("data pointer" in line or "storage" in line), line


def _stub(tmp_path):
    (tmp_path / "stub.c").write_text("int status, calls;\n" + "".join(f"int fp8_{n}(void) {{ ++calls; return status; }}\n" for n in CALLS))
    out = str(tmp_path / "stub.so")
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", out, str(tmp_path / "stub.c")], check=True)
    return f"""
import ctypes
stub = ctypes.CDLL({out!r}, ctypes.RTLD_GLOBAL)
status, calls = ctypes.c_int.in_dll(stub, "status"), ctypes.c_int.in_dll(stub, "calls")
F._invoke = lambda *a: print('again', a[0], flush=True)
"""


def test_a_hip_error_is_raised_and_the_call_is_not_made_again(tmp_path):
    code = _stub(tmp_path) + MORE + TRY + "status.value = -6\n"
    out = _run(code + "".join(f"attempt({n!r}, lambda: {c.format(s=0)})\n" for n, c in CALLS.items()) + "print(calls.value)\n")
    assert out[-1] == str(len(CALLS)) and len(out) == len(CALLS) + 1, out
    for line, name in zip(out, CALLS):
        assert line.startswith(f"{name} Fp8dsError FP8DS_ERR_HIP"), line


def test_a_refusal_is_left_to_the_bindings_checks(tmp_path):
    code = _stub(tmp_path) + MORE + TRY + "status.value = -3\n"
    out = _run(code + "".join(f"attempt({n!r}, lambda: {c.format(s=0)})\n" for n, c in CALLS.items()))
    assert out == [x for n in CALLS for x in (f"again fp8_{n}", f"{n} returned")], out
