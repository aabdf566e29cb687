"""The calls for drafted tokens near the ends of their ranges: vocabularies whose sums take more
than one round of a block's threads (above 131072 tokens), the largest number of sequences, nodes
and drafts."""
import numpy as np
import pytest
import torch

import oracle as O
from test_gpu_draft_verify import F, chain_case, check_chain, check_tree, tree_case  # noqa: F401
from test_gpu_tree_attend import Case

pytestmark = pytest.mark.gpu
WIDE = [131072, 131073, 151936, 262144, 262145]


@pytest.mark.parametrize("V", WIDE)
def test_wide_vocabularies(F, V):
    """Draws all along the row, chain and tree."""
    B = 9
    c = list(chain_case(B, 1, V, V % 7))
    c[4] = np.linspace(0, 1, B, dtype=np.float32)
    c[4][-1] = np.nextafter(np.float32(1), np.float32(0))
    for u in (0.0, 0.999):                        # accepted: from the target; refused: from the rest
        c[3][:] = u
        check_chain(F, *c[:3], None, *c[3:])
    c = list(tree_case(B, 3, V, V % 7))
    c[4] = np.linspace(0, 1, B, dtype=np.float32)
    c[4][-1] = np.nextafter(np.float32(1), np.float32(0))
    check_tree(F, *c[:3], None, *c[3:])


@pytest.mark.parametrize("V", WIDE)
def test_few_weights_in_a_wide_vocabulary(F, V):
    """Rows whose only weights lie in one round of the sums or another: the first and the last
    token, either side of a round's end, rounds without any."""
    spots = [[0], [V - 1], [131071], [0, V - 1], [5, 131071, 131072 % V], [131072 % V], [511, 512], [130000, V - 1],
             [1, 2, V - 2], []]
    r = [0.0, 0.3, 0.5, 0.75, 0.999, np.nextafter(np.float32(1), np.float32(0))]
    target = np.zeros((len(spots) * len(r), 2, V), np.float32)
    for i, s in enumerate(spots):
        for j in range(len(r)):
            for k, v in enumerate(s):
                target[i * len(r) + j, :, v] = 0.125 * (k + 1)
    draft = np.zeros((len(target), 1, V), np.float32)
    draft[:, 0, 3] = 1.0                          # token 3 has no weight: it is refused
    tok, u = np.full((len(target), 1), 3), np.full((len(target), 1), 0.5, np.float32)
    check_chain(F, target, draft, tok, None, u, np.array(r * len(spots), np.float32))
    # the root's child holds the row's first weight and is not taken: the others are drawn from,
    # or that row itself where there are none
    tok = np.zeros((len(target), 2), np.int64)
    for i, s in enumerate(spots):
        tok[i * len(r):(i + 1) * len(r), 1] = s[0] if s else 0
    check_tree(F, target, tok, np.tile([-1, 0], (len(target), 1)), None, np.ones((len(target), 2), np.float32),
               np.array(r * len(spots), np.float32))


def test_the_longest_chain_and_most_sequences(F):
    c = chain_case(2, 1024, 40, 1)
    c[3][:] *= 0.01                               # most are accepted
    check_chain(F, *c[:3], None, *c[3:])
    c = chain_case(16384, 2, 5, 2)
    check_chain(F, *c[:3], None, *c[3:])
    c = tree_case(16384, 3, 5, 2)
    check_tree(F, *c[:3], None, *c[3:])


@pytest.mark.parametrize("kind,Hq,Hkv,T,dh", [
    ("bf16", 8, 1, 8, 128),                       # 64 rows: the fewest stages that the rings have
    ("bf16", 1, 1, 1, 64), ("fp8", 8, 1, 8, 128), ("fp8", 3, 1, 3, 64), ("f32", 2, 1, 2, 64)])
def test_the_most_sequences_of_attention(F, kind, Hq, Hkv, T, dh):
    B, N = 1024, 272
    c = Case(kind, B, N, Hq, Hkv, dh, T, [(b * 37) % (N - T + 1) for b in range(B)],
             nodes=[T - b % 2 if b % 11 else 0 for b in range(B)], seed=18).dev(F)
    c.call(F)
    assert F.fdllm_get_status(c.ws) == F.OK
    c.check(seqs=[0, 1, 2, 511, 512, 1000, 1022, 1023])
