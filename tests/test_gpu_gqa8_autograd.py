"""What autograd learns of the grouped-query cache's calls."""
import pytest
import torch

import bit_kv_cache_nvfp4_gb300 as kv
import gqa8_ref as ref
from test_gpu_gqa8 import BF16, call_args, dev, ints

pytestmark = pytest.mark.gpu


def test_tensors_that_are_written_count_it():
    """So that a backward pass over something saved of them fails instead of
    using what they hold now."""
    device = dev()
    calls = call_args(device)
    err = torch.zeros(1, dtype=torch.int32, device=device)
    for f, names in (("append", ["pool", "scales"]), ("read", ["k_out", "v_out"]), ("attention", ["out", "lse"])):
        fn, args = calls[f]
        args = dict(args, dev_err=err)
        if f != "append":
            args.update(zip(names, (t.clone() for t in fn(**args))))
        if f == "attention":
            args["workspace"] = torch.empty(kv.attention_gqa8_workspace(2, 3, 5, 4, 2, 64), dtype=torch.uint8, device=device)
            names = names + ["workspace"]
        names = names + ["dev_err"]
        before = {n: t._version for n, t in args.items() if isinstance(t, torch.Tensor)}
        fn(**args)
        for n, was in before.items():
            assert args[n]._version == was + (1 if n in names else 0), (f, n)
    fn, args = calls["append"]
    before = args["pool"]._version
    with pytest.raises(ValueError):
        fn(**{**args, "v": args["v"][:4]})
    assert args["pool"]._version == before


def test_backward_over_an_overwritten_output_is_refused():
    device = dev()
    fn, args = call_args(device)["attention"]
    out, lse = (t.clone() for t in fn(**args))
    w = torch.ones_like(out, requires_grad=True)
    loss = (w * out).sum()                                       # saves out
    fn(**args, out=out, lse=lse)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


@torch.inference_mode()
def test_inference_tensors():
    device = dev()
    for fn, args in call_args(device).values():
        fn(**args)
    c = ref.Cache([100], 1, 64, device, seed=1)
    out, lse = torch.empty(1, 2, 64, dtype=BF16, device=device), torch.empty(1, 2, device=device)
    x = torch.randn(1, 2, 64, device=device).to(BF16)
    got = kv.attention_gqa8(x, c.pool, c.scales, c.page_table, c.seq_lens, ints([0, 1], device), 1, 0.1, out=out, lse=lse)
    assert got[0] is out and got[1] is lse


def test_results_carry_no_gradient():
    device = dev()
    fn, args = call_args(device)["attention"]
    out, lse = fn(**{**args, "q": args["q"].clone().requires_grad_()})
    assert not out.requires_grad and not lse.requires_grad
    want = fn(**args)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    fn, args = call_args(device)["append"]
    fn(**{**args, "k": args["k"].clone().requires_grad_()})
    assert not args["pool"].requires_grad
