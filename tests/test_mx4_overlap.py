"""Whether an output shares memory with the experts' matrices: found without a
look at every expert where they lie apart."""

import pytest
import torch

import sparse_dense_matmul_amd as sdm
from helpers import need_gpu
from sparse_dense_matmul_amd import mx4
from sparse_dense_matmul_amd.selection import _region


def refused(out, m):
    try:
        mx4._experts_apart("out", _region(out, out.stride(0)), [("gate", m)])
    except ValueError as e:
        return str(e)
    return ""


def test_rows_of_experts():
    base = torch.zeros(5, 12, 40, dtype=torch.bfloat16)
    halves = base[:, :4, 3:35], base[:, 4:8, 3:35]
    for m in halves:
        assert refused(m[2, 1:3, 5:9], m) == "out must not overlap gate[2]"
        assert refused(base[4, 0:12:11], m) == ("out must not overlap gate[4]" if m is halves[0] else "")
        # rows after each expert's, columns beside them, the other half, memory elsewhere
        assert not refused(base[3, 8:], m) and not refused(base[0, :, 35:], m) and not refused(base[0, :, :3], m)
        assert not refused(torch.zeros(2, 9, dtype=torch.bfloat16), m)
    assert not refused(halves[0][1], halves[1]) and not refused(halves[1][1], halves[0])
    assert refused(base[1, 2:5], base) == "out must not overlap gate"
    assert not refused(base[1, 2:5], base[:0]) and not refused(base[1, 2:5], base[:, :, :0])


def test_one_look_where_all_lies_apart(monkeypatch):
    looks = []
    real = mx4._overlap
    monkeypatch.setattr(mx4, "_overlap", lambda *a: looks.append(a) or real(*a))
    both = torch.zeros(400, 8, 16)
    mx4._experts_apart("out", _region(torch.zeros(2, 16), 16), [("gate", both[:, :4]), ("up", both[:, 4:])])
    assert len(looks) == 2


@pytest.mark.gpu
@pytest.mark.parametrize("weights", ["bf16", "mx4"])
def test_layer_over_views(weights):
    dev = need_gpu()
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=dev)  # noqa: E731
    if weights == "mx4":
        q = lambda n, r, k: sdm.Mx4(torch.zeros(n, r, k // 2, dtype=torch.uint8, device=dev),  # noqa: E731
                                    torch.zeros(n, r, k // 32, dtype=torch.uint8, device=dev), k)
        both, down = q(3, 64, 32), q(3, 32, 32)
        gate, up = (sdm.Mx4(both.codes[:, s], both.scales[:, s], 32) for s in (slice(32), slice(32, 64)))
        inside = both.codes[1].view(torch.bfloat16).view(-1, 32)[:4]
        name = "gate.codes"
    else:
        both, down = b(3, 64, 32), b(3, 32, 32)
        gate, up, inside, name = both[:, :32], both[:, 32:], both[2, 60:], "up"
    args = (b(4, 32), torch.zeros(4, 2, dtype=torch.int64, device=dev), torch.ones(4, 2, device=dev), gate, up, down)
    with pytest.raises(ValueError, match=f"out must not overlap {name}"):
        sdm.expert_mlp(*args, out=inside)
    ws = torch.zeros(sdm.expert_mlp_workspace(4, 2, 3, 32, 32), dtype=torch.uint8, device=dev)
    assert sdm.expert_mlp(*args, out=b(4, 32), workspace=ws).shape == (4, 32)
