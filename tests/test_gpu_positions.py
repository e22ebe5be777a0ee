"""Rows whose position lies past the rope table: the fused decode calls skip and report them, and attend no query that an
earlier call left in the workspace in their place."""
import pytest
import torch

from paged_gqa_decode_step_gb300 import workloads as wl

from gpu_util import TOL, binding, gpu_params, rope_tables_for

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

POSITIONS = (100, 5, 200, 70, 127, 128)          # rows 2 and 5 lie past a table of 128


@pytest.mark.parametrize("rows", [6, 606])        # the one-pass planner's calls, and longer ones
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("call", ["fused", "layers", "noalloc"])
def test_a_row_past_the_rope_table_is_skipped(call, dtype, rows):
    b = binding()
    w = wl.Workload("past_rope", rows, 8, 2, 64, 4, dtype, rope_theta=10000.0, positions="fixed",
                    fixed_positions=POSITIONS * (rows // 6))
    d = {k: v.cuda() for k, v in wl.generate(w, "cpu").items()}
    p = gpu_params(b, w, d["k_pool"].shape[0], rope_tables_for(b, w))
    ws = torch.zeros(max(b.workspace_size(p), b.layers_workspace_size(p, 1)), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(d["q"])

    def step():
        args = d["q"], d["k_new"], d["v_new"], d["positions"], d["table"], d["k_pool"], d["v_pool"], out
        if call == "fused":
            b.decode_fused(p, *args, ws)
        elif call == "noalloc":
            b.decode_fused_noalloc(p, *args)
        else:
            layer = dict(q=d["q"], k_new=d["k_new"], v_new=d["v_new"], k_pool=d["k_pool"], v_pool=d["v_pool"], out=out)
            b.decode_layers(p, [layer], d["positions"], d["table"], ws)
        torch.cuda.synchronize()

    step()
    b.check_status(ws)
    full, pools = out.clone(), [d[k].clone() for k in ("k_pool", "v_pool")]
    past = d["positions"] >= 128
    out.fill_(7.0)
    d["k_new"][past] += 1.0                        # shows in the pools if it is written
    p.rope_len = 128
    step()
    if call != "noalloc":
        with pytest.raises(b.PdattnError) as e:
            b.check_status(ws)
        assert e.value.status == b.EBADPOS
    assert (out[past] == 7).all()
    assert (out[~past].float() - full[~past].float()).abs().max() <= 2 * TOL[dtype][0]
    for k, pool in zip(("k_pool", "v_pool"), pools):
        assert torch.equal(d[k], pool)
