"""spec_sample's settings as numbers, as tensors of one element (the number they hold, as ever) and as
tensors with an entry for each row."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rejection_sampling_verify_02_amd as sv
    sv.load_library()
    return torch.device("cuda:0")


@pytest.mark.parametrize("B", [1, 3])
def test_tensors_of_one_element_are_numbers(dev, B):
    import torch
    import rejection_sampling_verify_02_amd as sv
    g = torch.Generator(device=dev).manual_seed(B)
    z = torch.randn((B, 5000), device=dev, generator=g) * 3
    u = torch.rand(B, device=dev, generator=g)
    want = sv.spec_sample(z, u, 0.8, 5)
    for T, k in ((torch.tensor([0.8]), torch.tensor([5])), (torch.tensor([[0.8]], dtype=torch.float64, device=dev), torch.tensor([[5]], device=dev)),
                 (torch.tensor(0.8), torch.tensor(5, device=dev)), (torch.tensor([0.8], device=dev), torch.tensor([5], device=dev)),
                 (0.8, torch.tensor([5], dtype=torch.int32))):
        got = sv.spec_sample(z, u, T, k)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # with what only the kernels of one temperature take
    got = sv.spec_sample(z, u, torch.tensor([0.8], device=dev), torch.tensor([5], dtype=torch.int32, device=dev), workspace=sv.Workspace())
    assert torch.equal(got[0], want[0])
    got = sv.spec_sample(z, None, torch.tensor([0.0], device=dev), torch.tensor([5]))
    assert torch.equal(got[0], z.argmax(1).int()) and not got[1].any()
    # among settings of other kinds
    want = sv.spec_sample(z, u, 0.8, 40, top_p=0.7, min_p=0.01)
    got = sv.spec_sample(z, u, torch.tensor([0.8]), torch.tensor([40]), top_p=torch.full((B,), 0.7, device=dev), min_p=torch.tensor([0.01], dtype=torch.float64))
    assert torch.equal(got[0], want[0]) and not got[1].any()


def test_tensors_of_another_size_are_refused(dev):
    import torch
    import rejection_sampling_verify_02_amd as sv
    z, u = torch.randn((3, 100), device=dev), torch.rand(3, device=dev)
    for n in (2, 4):
        with pytest.raises(ValueError):
            sv.spec_sample(z, u, torch.ones(n, device=dev))
        with pytest.raises(ValueError):
            sv.spec_sample(z, u, 1.0, top_p=torch.ones(n, device=dev))
    with pytest.raises(ValueError):
        sv.spec_sample(z, u, torch.ones(3))


def test_one_row_settings_under_capture(dev):
    """B = 1: a float32 (int32) tensor of the device is the row's setting, read when a graph is replayed."""
    import torch
    import rejection_sampling_verify_02_amd as sv
    z, u = torch.randn((1, 3000), device=dev) * 2, torch.tensor([0.6], device=dev)
    T, k = torch.tensor([0.7], device=dev), torch.tensor([30], dtype=torch.int32, device=dev)
    sv.spec_sample(z, u, T, k)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tok, st = sv.spec_sample(z, u, T, k)
    for t, n in ((0.7, 30), (1.5, 0), (0.7, 30)):
        T.fill_(t)
        k.fill_(n)
        g.replay()
        eager = sv.spec_sample(z, u, t, n, top_p=1.0 - 2.0 ** -24)
        torch.cuda.synchronize(dev)
        assert not st.any() and torch.equal(tok, eager[0])
