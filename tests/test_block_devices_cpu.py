"""The binding refuses tensors that no kernel can reach, before it gives their addresses away."""
import pytest
import torch

from output_centric_expert_gb300 import block_ops

BF16 = dict(dtype=torch.bfloat16)
INT = dict(dtype=torch.int32)


class OnGpu(torch.Tensor):
    """A tensor on the CPU that says it is on a GPU: what is left to refuse are the others."""

    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return 0


def _gpu(t):
    return t.as_subclass(OnGpu)


def _refuses(call, args, spoiled):
    """The call with `spoiled` of its arguments on the CPU raises, and reaches no kernel."""
    args = {k: v if k in spoiled or not isinstance(v, torch.Tensor) else _gpu(v) for k, v in args.items()}
    with pytest.raises(ValueError, match="on a GPU"):
        call(**args)


@pytest.mark.parametrize("spoiled", ["weights", "x", "y"])
def test_matvec(spoiled):
    w = block_ops.Fp4Weights(16, 64, device="cpu")
    w._on_gpu = spoiled != "weights"
    _refuses(block_ops.wd_fp4_matvec, dict(weights=w, x=torch.zeros(2, 64, **BF16), y=torch.zeros(2, 16)), [spoiled])


def test_packing():
    codes, scales = torch.zeros(16, 32, dtype=torch.uint8), torch.zeros(16, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="codes: not on a GPU"):
        block_ops.Fp4Weights.from_codes(codes, scales)
    with pytest.raises(ValueError, match="scales: not on a GPU"):
        block_ops.Fp4Weights.from_codes(_gpu(codes), scales)
    with pytest.raises(ValueError, match="w: not on a GPU"):
        block_ops.Fp4Weights.quantize(torch.zeros(16, 64))


@pytest.mark.parametrize("spoiled", ["cache", "k", "v", "block_table", "seq_lens", "cu_new", "err_flag"])
@pytest.mark.parametrize("fn", ["wd_kv4_append", "wd_kv4_gather"])
def test_cache_writers(fn, spoiled):
    c = block_ops.Kv4Cache(2, 16, 1, 64, device="cpu")
    c._on_gpu = spoiled != "cache"
    k, v = ("k_out", "v_out") if fn == "wd_kv4_gather" else ("k", "v")
    _refuses(getattr(block_ops, fn), {"cache": c, k: torch.zeros(1, 1, 64, **BF16), v: torch.zeros(1, 1, 64, **BF16),
                                      "block_table": torch.zeros(1, 2, **INT), "seq_lens": torch.zeros(1, **INT),
                                      "cu_new": torch.zeros(2, **INT), "err_flag": torch.zeros(1, **INT)},
             [{"k": k, "v": v}.get(spoiled, spoiled)])


@pytest.mark.parametrize("spoiled", ["cache", "q", "block_table", "seq_lens", "out", "workspace", "lse", "err_flag"])
def test_attend(spoiled):
    c = block_ops.Kv4Cache(2, 16, 1, 64, device="cpu")
    c._on_gpu = spoiled != "cache"
    _refuses(block_ops.wd_kv4_attend, dict(
        cache=c, q=torch.zeros(1, 2, 64, **BF16), block_table=torch.zeros(1, 2, **INT), seq_lens=torch.zeros(1, **INT),
        out=torch.zeros(1, 2, 64, **BF16), workspace=torch.zeros(16, dtype=torch.uint8), lse=torch.zeros(1, 2),
        err_flag=torch.zeros(1, **INT)), [spoiled])


@pytest.mark.parametrize("spoiled", ["res", "res_out", "out", "y", "w_post", "gate", "w_pre"])
def test_norm(spoiled):
    rows = {n: torch.zeros(2, 64) for n in ("res", "res_out", "out", "y")}
    _refuses(block_ops.wd_block_norm, dict(rows, w_post=torch.zeros(64), w_pre=torch.zeros(64), gate=torch.zeros(1, 64)), [spoiled])


def test_an_error_flag_has_an_element_and_a_workspace_is_dense():
    with pytest.raises(ValueError, match="err_flag"):
        block_ops._flag(_gpu(torch.zeros(0, **INT)))
    c = block_ops.Kv4Cache(2, 16, 1, 64, device="cpu")
    c._on_gpu = True
    with pytest.raises(ValueError, match="contiguous"):
        block_ops.wd_kv4_attend(c, _gpu(torch.zeros(1, 2, 64, **BF16)), _gpu(torch.zeros(1, 2, **INT)), _gpu(torch.zeros(1, **INT)),
                                _gpu(torch.zeros(1, 2, 64, **BF16)), _gpu(torch.zeros(64, dtype=torch.uint8)[::2]))
