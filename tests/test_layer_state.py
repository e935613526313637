"""What LogicalEP keeps between calls when its layer changes, without a GPU:
graphs captured before do not outlive the buffers that they read and write."""
import pytest
import torch

from combine_topk_ids_dest_amd.emulate import LogicalEP


def _ep(**kw):
    return LogicalEP(T=4, H=64, E=8, K=2, W=2, cap=4, row_bytes=[128],
                     combine_dtype=torch.bfloat16, device="cpu", **kw)


def _weights(seed=0):
    g = torch.Generator().manual_seed(seed)
    return dict(w13=torch.randn(8, 64, 64, generator=g).bfloat16(),
                w2=torch.randn(8, 64, 32, generator=g).bfloat16())


class _Graph:
    replays = 0

    def replay(self):
        _Graph.replays += 1


def test_step_graphs_needs_a_capture():
    with pytest.raises(RuntimeError, match="capture_lane_graphs"):
        _ep().step_graphs([None])


@pytest.mark.parametrize("layers", [0, 1])
def test_a_new_layer_drops_the_captured_graphs(layers):
    """With a layer the graphs hold its buffers' addresses; without one they
    run the path without the layer that was set since."""
    ep = _ep()
    for i in range(layers):
        ep.set_layer(**_weights(i))
    ep._lane_graphs = [[_Graph()] for _ in range(3)]          # as a capture leaves them
    ep.set_layer(**_weights(7))
    with pytest.raises(RuntimeError, match="capture_lane_graphs"):
        ep.step_graphs([None])
    assert _Graph.replays == 0


def test_a_refused_layer_leaves_the_graphs():
    ep = _ep()
    ep.set_layer(**_weights())
    graphs = ep._lane_graphs = [[_Graph()] for _ in range(3)]
    with pytest.raises(ValueError):
        ep.set_layer(**dict(_weights(), shared13=torch.zeros(8, 64).bfloat16()))
    assert ep._lane_graphs is graphs


def test_a_fused_step_with_a_layer_is_refused_before_anything_is_enqueued():
    ep = _ep()
    ep.set_layer(**_weights())
    graphs = ep._lane_graphs = [[_Graph()] for _ in range(3)]
    calls = []
    ep._prepared = lambda kind, i: calls.append(kind) or (lambda stream: None)
    for refused in (lambda: ep.step(fused_local=True),
                    lambda: ep.step(fused_local=True, streams=[None]),
                    lambda: ep.capture_lane_graphs(fused_local=True)):
        with pytest.raises(ValueError, match="share one buffer"):
            refused()
    assert calls == [] and ep._lane_graphs is graphs


@pytest.mark.parametrize("E,H,inter", [(8, 384, 128), (8, 256, 384), (16, 640, 640), (8, 512, 128)])
def test_every_rank_s_block_scales_start_aligned(E, H, inter):
    """The fp8 product takes block scales from a 16-byte boundary on; with an odd
    number of blocks an expert, a rank's slice of dense scales starts at 4, 8 or
    12 bytes."""
    ep = LogicalEP(T=4, H=H, E=E, K=2, W=8, cap=4, row_bytes=[2 * H], combine_dtype=torch.bfloat16,
                   device="cpu", quant_group=128)
    s13 = torch.rand(E, 2 * (-(-inter // 128)), H // 128)
    s2 = torch.rand(E, H // 128, inter // 128)
    f8 = torch.float8_e4m3fn
    ep.set_layer(torch.zeros(E, 2 * inter, H, dtype=f8), torch.zeros(E, H, inter, dtype=f8), s13, s2)
    per = E // 8
    for name, given in (("w13_scale", s13), ("w2_scale", s2)):
        for r in range(8):
            mine = ep._layer[name][r * per:(r + 1) * per]
            assert mine.data_ptr() % 16 == 0, (name, r)
            assert torch.equal(mine, given[r * per:(r + 1) * per])
            assert mine[0].is_contiguous()


@pytest.mark.gpu
def test_graphs_of_a_new_layer_run_the_new_layer():
    from test_gpu_layer import ROUTE, build, check, weights
    ep, xs, d, f13, f2 = build(4, 16, 3, 60, 256, 128, 64, False, lanes=2)
    streams = [torch.cuda.Stream() for _ in range(2)]
    ep.capture_lane_graphs()
    ep.step_graphs(streams)
    torch.cuda.synchronize()
    check(ep, xs, d, f13, f2, False)
    d, f13, f2 = weights(16, 256, 192, 40, False, seed=9)
    ep.set_layer(route=ROUTE, **{k: v.cuda() for k, v in d.items()})
    with pytest.raises(RuntimeError, match="capture_lane_graphs"):
        ep.step_graphs(streams)
    ep.capture_lane_graphs()
    for _ in range(3):
        ep.out.fill_(0)
        torch.cuda.synchronize()
        ep.step_graphs(streams)
        torch.cuda.synchronize()
        check(ep, xs, d, f13, f2, False)


@pytest.mark.gpu
def test_layer_with_an_odd_number_of_block_scales_a_rank():
    from test_gpu_layer import build, check
    ep, *rest = build(8, 8, 2, 40, 384, 128, 64, True)
    ep.step()
    torch.cuda.synchronize()
    check(ep, *rest, True)
