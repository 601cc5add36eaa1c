"""What the header promises of attention's workspace and of its bits."""
import pytest
import torch

from test_gpu_attend import LAYOUTS, History, Located, dhs  # noqa: F401

pytestmark = pytest.mark.gpu


def bound(lay):
    return 512 * (lay.value + 2) * torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("name", ["latent", "latent_128", "grouped", "largest", "smallest"])
def test_workspace_bound(dhs, name):  # noqa: F811
    lay = LAYOUTS[name]
    env = Located(dhs, lay)
    loc = env.rand_loc(1, 1)
    most = 0
    for Q in (1, 3, 8, 64):
        for k in (1, 129, 700, 2048, 5000, 40000, 300000):
            for n in (1, 2, 7, 60, 260):
                it, t = env.item(loc)
                it.queries, it.topk = Q, k
                st, keep = dhs.make_attend([it] * n, **lay.args())
                most = max(most, env.pool.attend_bytes(st))
    assert 0 < most <= bound(lay)


def test_one_workspace_while_a_history_grows(dhs):  # noqa: F811
    """Appends take the history from no parts to many; the workspace stays."""
    lay = LAYOUTS["grouped"]
    work = torch.empty(bound(lay), dtype=torch.uint8, device="cuda")
    for appended in (0, 140, 1500):
        env = History(dhs, lay, [500, 3], T=64, appended=appended, seed=1)
        its = env.items(1)
        st, keep = dhs.make_attend([it for it, _ in its], **lay.args())
        st.work_dev, st.work_bytes = work.data_ptr(), work.numel()
        assert env.pool.attend(st) == 0
        env.check(its, 1)


@pytest.mark.parametrize("name", ["latent", "grouped"])
def test_the_same_step_gives_the_same_bits(dhs, name):  # noqa: F811
    env = Located(dhs, LAYOUTS[name], seed=3)
    items, keeps = [], []
    for Q, k in ((1, 3000), (3, 200), (2, 777), (1, 0)):
        it, t = env.item(env.rand_loc(Q, k))
        items.append(it)
        keeps.append(t)
    st, keep = dhs.make_attend(items, **env.lay.args())
    work = torch.empty(bound(env.lay), dtype=torch.uint8, device="cuda")
    st.work_dev, st.work_bytes = work.data_ptr(), work.numel()
    outs = [o for t in keeps for o in t[1:3]]
    first = None
    for fill in (0, 255, 7):
        work.fill_(fill)
        assert env.pool.attend(st) == 0
        torch.cuda.synchronize()
        if first is None:
            first = [o.clone() for o in outs]
        assert all(torch.equal(a, b) for a, b in zip(first, outs))
