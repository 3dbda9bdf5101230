"""The binding loads where PyTorch is absent: the library's C entries and sizes are
there, and a call on tensors says what it misses."""
import subprocess
import sys

CODE = """
import sys
sys.modules["torch"] = None          # what an import of an absent module meets
import block_quantized_expert_gb300 as bqe
lib = bqe.load_library()
assert all(hasattr(lib, n) for n in bqe.EXPORTS)
assert bqe.moe_workspace_bytes(bqe.MoeConfig(256, 128, 16, 2, 4)) > 0
assert bqe.moe_permute_scratch_bytes(4, 2, 16) > 0
assert lib.moe_dispatch(None, 7, 0, 1, 1, 1, None, 1, None, None, 0, None) == bqe.MOE_ERR_INVALID_ARG
assert "dtype" in bqe.moe_last_error()
try:
    bqe.moe_check_product()
except ModuleNotFoundError as e:
    assert "torch" in str(e)
else:
    raise AssertionError("no error")
print("fine")
"""


def test_binding_loads_without_torch():
    r = subprocess.run([sys.executable, "-c", CODE], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr


def test_a_broken_torch_is_not_hidden(tmp_path):
    (tmp_path / "torch.py").write_text("import no_such_module_of_torch\n")
    code = f"import sys; sys.path.insert(0, {str(tmp_path)!r}); import block_quantized_expert_gb300"
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode != 0 and "no_such_module_of_torch" in r.stderr
