"""The dropout's generator: an implementation on arbitrary counter and key words, held to the
published known answers of Philox4x32-10, and the kernels' masks held to it."""
import numpy as np
import pytest
import torch

M32 = 0xFFFFFFFF


def philox(counter, key):
    """The four output words for four counter words and two key words, in Python's integers."""
    c, k = list(counter), list(key)
    for _ in range(10):
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & M32, (p0 >> 32) ^ c[3] ^ k[1], p0 & M32]
        k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
    return c


@pytest.mark.parametrize("counter,key,words", [
    ([0] * 4, [0] * 2, [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
    ([M32] * 4, [M32] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
     [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1])])
def test_published_known_answers(counter, key, words):
    """All zeros, all ones, and the digits of pi, where no two words are alike."""
    assert philox(counter, key) == words


def numbers(block, step, seed):
    """The eight 16-bit numbers of a block by the operators' definition: counter (block low, block
    high, step low, step high), key (seed low, seed high), words low half first."""
    w = philox([block & M32, block >> 32, step & M32, step >> 32], [seed & M32, seed >> 32])
    return [x for v in w for x in (v & 0xFFFF, v >> 16)]


SEEDS = [(0, 0), ((1 << 64) - 1, (1 << 64) - 1), (0x299F31D0A4093822, 0x0370734413198A2E), (1, 1 << 32), (1 << 32, 1), (5, 6)]


def test_other_references_read_the_words_alike():
    """The vectorised references of the operators' tests against this one, every word different."""
    from test_ops_gpu import philox as blocks_from_zero
    from test_ops_layers_gpu import _philox_at
    for seed, step in SEEDS:
        got = blocks_from_zero(seed, step, 5)
        assert got.tolist() == [numbers(b, step, seed) for b in range(5)]
    at = np.array([0, 1, 0x85A308D3, 1 << 32, 0x85A308D3243F6A88 >> 31], dtype=np.uint64)
    assert _philox_at(at, 5, 6).tolist() == [numbers(int(b), 6, 5) for b in at]


@pytest.mark.gpu
@pytest.mark.parametrize("seed,step", SEEDS)
def test_masks_of_the_kernels(seed, step):
    """dropout and gated_act keep what the definition keeps, for thresholds on both sides of the
    numbers that were drawn."""
    import mixture_experts_layer_46_amd as M
    print(f"masks seed={seed:x} step={step:x}", flush=True)
    n = 8 * 40
    u = torch.tensor([x for b in range(n // 8) for x in numbers(b, step, seed)])
    one = torch.ones(n, dtype=torch.float32, device="cuda")
    for t in sorted({1, 32768, int(u[17]), int(u[17]) + 1, int(u[250]), 65535}):
        if t == 0:
            continue
        want = u >= t
        assert torch.equal(M.dropout(one, t / 65536, seed, step).cpu() != 0, want)
        assert torch.equal(M.gated_act(one.view(4, 80), None, t / 65536, seed, step).cpu().view(-1) != 0, want)
