"""The package is imported without torch, as before it had operators on tensors;
these come when they are named."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAMES = ("MXMatrix", "PreferenceLoss", "clip_grad_norm", "mx_matmul", "mx_quantize", "preference_loss",
         "preference_loss_backward")


def _run(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_import_does_not_bring_torch():
    _run("import sys; import hash_table_cache_gb300 as hkv; assert 'torch' not in sys.modules\n"
         f"assert set({NAMES!r}) | {{'operators', 'HashTable'}} <= set(dir(hkv))")


def test_import_and_the_c_layer_work_without_torch():
    _run("import sys; sys.modules['torch'] = None\n"
         "from hash_table_cache_gb300 import _build\n_build.build()\n"
         "import hash_table_cache_gb300 as hkv\n"
         "assert hkv.hkv_status_string(0) == 'ok' and hkv.hkv_get_wait_timeouts")


def test_operators_come_when_named():
    each = "".join(f"assert hkv.{n} is hkv.operators.{n}\n" for n in NAMES)
    _run(f"import hash_table_cache_gb300 as hkv\n{each}")
    _run(f"from hash_table_cache_gb300 import {', '.join(NAMES)}")
    _run("import hash_table_cache_gb300 as hkv; hkv.operators.mx_matmul; hkv.mx_matmul")
    _run("import hash_table_cache_gb300.operators as o; import hash_table_cache_gb300 as h; assert h.operators is o")
    _run("import hash_table_cache_gb300 as hkv\ntry:\n    hkv.nothing\nexcept AttributeError as e:\n"
         "    assert 'nothing' in str(e)\nelse:\n    raise SystemExit(1)")
