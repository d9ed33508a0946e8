"""The two bindings' checks of the operators beside the FP8 attention."""

import pytest
import torch

import int4_token_head_gb300 as kv
from int4_token_head_gb300 import _lib
from test_fp8_gpu import _changed

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("op", ["axes", "shared", "mass", "evict"])
def test_both_bindings_refuse_the_same_calls(monkeypatch, op):
    """Every argument changed in turn, in calls without tokens or sequences (nothing is launched): through the call
    module and through ctypes the same outcome."""
    assert _lib._calls() is not _lib._Calls
    d, cuda = 64, dict(device="cuda")
    cache = [torch.zeros(4, 16, 2, d, dtype=torch.uint8, **cuda).view(torch.float8_e4m3fn) for _ in range(2)] + [
        torch.ones(4, 2, **cuda) for _ in range(2)]
    ints = lambda *shape: torch.zeros(*shape, dtype=torch.int32, **cuda)
    n = 0 if op == "evict" else 3
    table, lens, start = ints(n, 5), ints(n), ints(n + 1)
    q, k = ([torch.zeros(0, h, d, dtype=torch.bfloat16, **cuda) for _ in range(2)] for h in (4, 2))
    lse, mass = torch.zeros(0, 4, **cuda), [torch.zeros(n, 2, 80, **cuda) for _ in range(2)]
    w = torch.ones(d, dtype=torch.bfloat16, **cuda)
    status = ints(1)
    f, args = {
        "axes": (kv.qk_norm_rope_axes, [q[0], k[0], torch.zeros(2, 0, dtype=torch.int64, **cuda), torch.ones(8, 32, **cuda),
                                        kv.rope_axes((8, 8)), w, w.clone(), 1e-6, q[1], k[1], False, status]),
        "shared": (kv.attention_fp8_shared, [q[0], *cache, table, lens, start, 3, 64, ints(2), ints(1), 3, 0.1, q[1],
                                             torch.zeros(64, dtype=torch.uint8, **cuda), lse, status]),
        "mass": (kv.attention_mass_fp8, [q[0], lse, cache[0], cache[2], table, lens, start, 3, 64, 0.1, mass[0], status]),
        "evict": (kv.evict_fp8, [*cache, mass[0], table, lens, 20, 4, ints(n, 2), mass[1], ints(n), ints(n, 2, 20), status]),
    }[op]

    def outcome(args):
        try:
            return f(*args)
        except Exception as e:
            return type(e), str(e)

    module, refused = _lib._calls(), 0
    assert outcome(args) is None
    for i, x in enumerate(args):
        others = [("text", "3"), ("none", None), ("half", 0.5), ("large", 1 << 40), ("bytes", b"\x01" * 16), ("short", b"\x01")]
        for what, y in _changed(x) if torch.is_tensor(x) else others:
            call = [*args[:i], y, *args[i + 1:]]
            monkeypatch.setattr(_lib, "_fp8", module)
            first = outcome(call)
            monkeypatch.setattr(_lib, "_fp8", _lib._Calls)
            assert outcome(call) == first, (i, what)
            refused += first is not None
    assert refused > 4 * len(args)
