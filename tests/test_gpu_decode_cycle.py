"""The example's decode cycles: cache writes, attention in prompt, draft and
verify passes, acceptance and commit, over either cache."""
import pytest
import torch

from tests.gpu_util import needs_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window,sinks", [(0, 0), (24, 2)])
@pytest.mark.parametrize("cache", ["bf16", "q4"])
def test_cycles_leave_the_cache_a_prompt_pass_would(cache, window, sinks):
    """After some cycles the committed slots hold what one pass over the whole
    sequences writes, so the next token's logits agree.

    The two ways differ in roundings alone (a pass's rows go through kernels of
    other shapes): bf16 results within one step of each other where sums are
    ordered differently, half a step (2^-8) for each of the at most 6 rounded
    tensors per layer and 2 layers on the way to logits of variance about 1,
    in relative mean square terms 12 * 2^-8; over the 4-bit cache a key or
    value that crosses a rounding boundary moves by a whole step, up to a
    third of itself, for the few that do: 4 times that."""
    ml = needs_gpu()
    from examples.decode_cycle import Model, decode
    k = 3
    prompts = [list(range(i, i + 3 + 11 * i)) for i in range(6)]
    adapter = torch.arange(6, device="cuda").int() % 4
    model = Model(cache=cache, window=window, sinks=sinks)
    out, kept = decode(model, prompts, adapter, k, 6, seed=3)
    assert model.status() == 0 and 0 <= kept <= 6 * 6 * k
    assert all(len(o) >= len(p) + 6 and o[:len(p)] == p for o, p in zip(out, prompts))

    again, kept_again = decode(model, prompts, adapter, k, 6, seed=3)     # the same from the same draws
    assert again == out and kept_again == kept

    for b, o in enumerate(out):
        seq = torch.zeros(1, dtype=torch.int32, device="cuda")
        blocks = (len(o) + 15) // 16
        one = adapter[b:b + 1]
        fresh = Model(cache=cache, window=window, sinks=sinks)
        table = torch.arange(blocks, device="cuda").int().view(1, blocks)
        tok = torch.tensor([o], device="cuda")
        whole = fresh.forward(tok, one, table, seq, 0, ml.VERIFY)[0, -1]
        other = Model(cache=cache, window=window, sinks=sinks)
        n = len(prompts[b])
        other.forward(tok[:, :n], one, table, seq, 0, ml.VERIFY)
        for p in range(n, len(o)):                                       # a row at a time
            step = other.forward(tok[:, p:p + 1], one, table, seq, p, ml.VERIFY)[0, -1]
        bound = 12 * 2.0 ** -8 * (4 if cache == "q4" else 1)
        assert float((step - whole).norm() / whole.norm()) <= bound
