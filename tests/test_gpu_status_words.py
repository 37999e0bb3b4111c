"""Status words are zeroed many at a time: whichever call made them, the next one gets a plain tensor of its own."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from tests.test_gpu_gather_tokens import cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from load_balanced_split_step_b200 import binding
    return binding


def calls(B):
    """One call the short way and one the long way; a stream of their own, so that both begin with no words in hand."""
    table = torch.tensor([[3, 0, -1], [1, -1, -1]], dtype=torch.int32, device="cuda")
    ref = torch.tensor([1, 1, 0, 1, 0, 0], dtype=torch.int32, device="cuda")
    (kp, vp), pages, seq, _, kw = cache(1, (5, 9), 2, 64, 16, "HND", "bf16")
    torch.cuda.synchronize()
    return {"short": lambda: B.compact_pages(table, ref).status, "long": lambda: B.gather_tokens(kp, vp, pages, seq, 14, **kw)[3]}


# (The long way makes its outputs by torch: in FakeTensorMode it takes none but the caller's.)
@pytest.mark.parametrize("mode,first", [(torch.inference_mode, "short"), (torch.inference_mode, "long"), (torch.no_grad, "short"),
                                        (torch.no_grad, "long"), (FakeTensorMode, "short")])
@pytest.mark.parametrize("then", ["short", "long"])
def test_words_do_not_keep_the_mode_that_made_them(B, mode, first, then):
    call = calls(B)
    with torch.cuda.stream(torch.cuda.Stream()):
        with mode():
            call[first]()
        for _ in range(3):
            st = call[then]()
            assert type(st) is torch.Tensor and not st.is_inference() and st.shape == (1,) and int(st.item()) == 0
            st.bitwise_or_(4)
            st.zero_()
    torch.cuda.synchronize()


def test_words_are_apart(B):
    call = calls(B)
    with torch.cuda.stream(torch.cuda.Stream()):
        words = [call["short"]() for _ in range(200)] + [call["long"]() for _ in range(100)]
        for i, w in enumerate(words):
            w.fill_(i)
        assert [int(w) for w in words] == list(range(300))
        assert all(not w._is_view() for w in words)
    torch.cuda.synchronize()
