"""The sequence-layer operators in a CUDA graph: captured once the workspace is there, replayed on new inputs."""
import pytest


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [3, 150])
def test_layer_in_a_graph(tokens):
    import torch

    import mixed_precision_refinement_gb300 as zs
    gen = torch.Generator("cuda").manual_seed(tokens)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    d, hk, hv, dk = 96, 2, 4, 32
    w, b = randn(d).bfloat16(), randn(d).bfloat16()
    wi, bi = randn(2 * hk * dk + hv * dk, d).bfloat16() / 10, randn(2 * hk * dk + hv * dk).bfloat16()
    x, g, beta = randn(tokens, d).bfloat16(), -randn(tokens, hv).abs(), torch.rand(tokens, hv, generator=gen, device="cuda")
    do, state = randn(tokens, hv, dk).bfloat16(), randn(1, hv, dk, dk)
    with zs.Seq() as s:
        def run():
            h, mean, rstd = s.layernorm(x, w, b)
            a, z = s.linear(h, wi, bi, act="gelu", keep=True)
            q, k, v = a.split([hk * dk, hk * dk, hv * dk], dim=1)
            q, k, v = q.unflatten(1, (hk, dk)) / 8, k.unflatten(1, (hk, dk)) / 8, v.unflatten(1, (hv, dk))
            o, last = s.delta(q, k, v, g, beta, state)
            grads = s.delta_bwd(do, q, k, v, g, beta, state)
            back = s.linear_bwd(a, h, wi, z, act="gelu") + s.layernorm_bwd(h, x, mean, rstd, w)
            return (h, a, o, last) + grads + back

        run()  # the workspace grows here
        held = zs.zsolve_seq_workspace_bytes(s.seq)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        for seed in range(2):  # other inputs in the same places
            x.copy_(randn(tokens, d).bfloat16())
            g.copy_(-randn(tokens, hv).abs())
            state.copy_(randn(1, hv, dk, dk))
            graph.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in out]
            for p, q in zip(got, run()):
                assert torch.equal(p, q)
        assert zs.zsolve_seq_workspace_bytes(s.seq) == held
        # a larger workspace leaves the graph its own
        zs.zsolve_seq_reserve(s.seq, 4 * held + (1 << 20))
        filler = torch.full((4 * held + (1 << 20),), 255, dtype=torch.uint8, device="cuda")
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(got, out):
            assert torch.equal(p, q)
        assert bool((filler == 255).all())
        zs.zsolve_seq_check(s.seq)


@pytest.mark.gpu
def test_capture_without_a_workspace_is_refused():
    import torch

    import mixed_precision_refinement_gb300 as zs
    q = torch.randn(100, 1, 16, device="cuda")
    g = -torch.rand(100, 1, device="cuda")
    with zs.Seq() as s:
        s.layernorm(q)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            with pytest.raises(zs.ZsolveError) as e:
                s.delta(q, q, q, g, -g)
            q.add(0)
        assert e.value.status == zs.ZSOLVE_ESTATE
        torch.cuda.synchronize()
        o, _ = s.delta(q, q, q, g, -g)  # outside the capture it grows
        assert bool(torch.isfinite(o).all())
