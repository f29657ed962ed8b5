"""CPU model of the signals inside a CTA pair of the many-rows expert kernel.

Every role of both CTAs is a generator, and the order of their steps is random; copies, MMAs and arrivals
complete later, the arrivals of one commit at the two CTAs independently of each other. Checked:
  * an MMA finds its k-block in both CTAs' rings and weight slots when it is issued and still when it
    completes;
  * an adding warp finds the group that it waits for;
  * no barrier is completed twice where a wait can tell only one phase from the next;
  * no arrival reaches a CTA that has left.
The counts, rings and waits are those of csrc/wq_experts_large.cu; a model whose second CTA leaves without
its wait for the last commits must break the last rule.
"""
import random

import pytest

STAGES, SLOTS = 8, 4
GATHER, TURNS, QUARTERS, ADDERS = 3, 2, 4, 3  # 16 adding warps act alike: three


class Fault(Exception):
    pass


class Barrier:
    def __init__(self, cta, count):
        self.cta, self.count, self.pending, self.phase = cta, count, count, 0

    def arrive(self):
        if self.cta["left"]:
            raise Fault("an arrival at a CTA that has left")
        self.pending -= 1
        if self.pending == 0:
            self.pending, self.phase = self.count, self.phase + 1

    def passed(self, n):
        """Whether phase n is complete; a wait by parity cannot tell n + 2 from n."""
        if self.phase > n + 1:
            raise Fault("a barrier is two phases ahead of a wait")
        return self.phase == n + 1


def run(seed, tiles, k_blocks, group_blocks, second_waits=True):
    """tiles of k_blocks; a group's sums cover group_blocks k-blocks, or a k-block has 1 / group_blocks groups."""
    rng = random.Random(seed)
    blocks = tiles * k_blocks
    per_block = round(1 / group_blocks) if group_blocks < 1 else 1
    groups = blocks * per_block if group_blocks <= 1 else tiles * (k_blocks // group_blocks)
    ctas = [{"left": False, "ring": [None] * STAGES, "slot": {}, "roles": 0} for _ in range(2)]
    for c in ctas:
        c["empty"] = [Barrier(c, 1) for _ in range(STAGES)]
        c["sum_full"] = [Barrier(c, 1) for _ in range(2)]
        c["drain"] = Barrier(c, 1)
    full = [Barrier(ctas[0], 2 + 2 * QUARTERS) for _ in range(STAGES)]
    sum_empty = [Barrier(ctas[0], 2 * ADDERS) for _ in range(2)]
    later = []     # (step at which it may happen, action)
    pipe = []      # the tensor pipe: MMAs and commits in order
    sums = [None, None]
    now = [0]

    def after(most, action, of_thread=False):
        later.append((now[0] + rng.randint(1, most), action, of_thread))

    def gather(c, w):
        pending = None
        for n in range(w, blocks, GATHER):
            while n >= STAGES and not c["empty"][n % STAGES].passed(n // STAGES - 1):
                yield
            done = {}

            def copied(n=n, done=done):
                c["ring"][n % STAGES] = n
                done["yes"] = True
            after(6, copied)
            yield
            if pending:
                while "yes" not in pending[1]:
                    yield
                after(4, full[pending[0] % STAGES].arrive, True)
            pending = (n, done)
        if pending:
            while "yes" not in pending[1]:
                yield
            after(4, full[pending[0] % STAGES].arrive, True)

    def dequant(c, turn, quarter):
        for n in range(turn, blocks, TURNS):
            while n >= SLOTS and not c["empty"][(n - SLOTS) % STAGES].passed((n - SLOTS) // STAGES):
                yield
            c["slot"][n % SLOTS, quarter] = n
            yield
            after(4, full[n % STAGES].arrive, True)

    def check(n, when):
        for c in ctas:
            if c["ring"][n % STAGES] != n or any(c["slot"].get((n % SLOTS, q)) != n for q in range(QUARTERS)):
                raise Fault(f"k-block {n} is not there {when}")

    def commit(names):
        def fire():
            for c in ctas:
                after(12, names(c).arrive)
        pipe.append(fire)

    def mma():
        m = in_group = 0
        for n in range(blocks):
            for _ in range(per_block):
                if in_group == 0:
                    while m >= 2 and not sum_empty[m & 1].passed((m >> 1) - 1):
                        yield
                while not full[n % STAGES].passed(n // STAGES):
                    yield
                check(n, "when it is issued")

                def mult(n=n, m=m):
                    check(n, "when its MMA completes")
                    sums[m & 1] = m
                pipe.append(mult)
                yield
                if group_blocks < 1:
                    commit(lambda c, m=m: c["sum_full"][m & 1])
                    m += 1
            commit(lambda c, n=n: c["empty"][n % STAGES])
            in_group += 1
            if group_blocks >= 1 and in_group == group_blocks:
                commit(lambda c, m=m: c["sum_full"][m & 1])
                m, in_group = m + 1, 0
            elif group_blocks < 1:
                in_group = 0
            yield
        commit(lambda c: c["drain"])

    def add(c):
        for m in range(groups):
            while not c["sum_full"][m & 1].passed(m >> 1):
                yield
            if sums[m & 1] != m:
                raise Fault(f"the sums of group {m} are not there")
            yield
            if sums[m & 1] != m:
                raise Fault(f"the sums of group {m} went while they were read")
            after(4, sum_empty[m & 1].arrive, True)

    roles = []
    for c in ctas:
        for r in ([gather(c, w) for w in range(GATHER)] + [dequant(c, t, q) for t in range(TURNS) for q in range(QUARTERS)] +
                  [add(c) for _ in range(ADDERS)] + ([mma()] if c is ctas[0] else [])):
            roles.append((c, r))
            c["roles"] += 1
    at_end = set()
    while not all(c["left"] for c in ctas):
        now[0] += 1
        if now[0] > 200000:
            raise Fault("the roles wait for one another")
        for item in [x for x in later if x[0] <= now[0]]:
            later.remove(item)
            item[1]()
        if pipe and rng.random() < 0.7:
            pipe.pop(0)()
        for c, r in rng.sample(roles, min(len(roles), 8)):
            try:
                next(r)
            except StopIteration:
                roles.remove((c, r))
                c["roles"] -= 1
        for i, c in enumerate(ctas):
            here = c["drain"].phase == 1 and all(b.phase == (blocks - s + STAGES - 1) // STAGES
                                                 for s, b in enumerate(c["empty"]))
            if c["roles"] == 0 and (here or (i == 1 and not second_waits)):
                at_end.add(i)
        # the cluster's barrier: what the CTAs' threads did before it, their arrivals too, is done behind it
        if len(at_end) == 2 and not any(of_thread for _, _, of_thread in later):
            for c in ctas:
                c["left"] = True
    for fire in pipe:
        fire()
    for _, action, _ in later:
        action()


SHAPES = [(1, 1, 1), (3, 1, 1), (2, 6, 1), (3, 5, 5), (2, 9, 9), (4, 6, 2), (2, 5, 0.5), (2, 3, 0.25), (5, 1, 0.25), (1, 24, 1)]


@pytest.mark.parametrize("tiles,k_blocks,group_blocks", SHAPES)
def test_the_pair_signals_in_order(tiles, k_blocks, group_blocks):
    for seed in range(60):
        run(seed, tiles, k_blocks, group_blocks)


@pytest.mark.parametrize("tiles,k_blocks,group_blocks", SHAPES)
def test_a_second_cta_that_does_not_wait_leaves_too_early(tiles, k_blocks, group_blocks):
    faults = 0
    for seed in range(200):
        try:
            run(seed, tiles, k_blocks, group_blocks, second_waits=False)
        except Fault as f:
            assert "has left" in str(f)
            faults += 1
    assert faults


def test_the_kernel_waits_in_both_ctas():
    # the wait stands behind the block barrier that all roles of a CTA come to, for either rank
    import os
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                            "bit_weight_quantized_prepack_b200", "csrc", "wq_experts_large.cu")).read()
    tail = src[src.index("cluster_sync();  // neither CTA leaves") - 1400:src.index("cluster_sync();  // neither CTA leaves")]
    tail = tail[tail.index("__syncthreads();"):]
    assert "wait_phase(&bars.drain" in tail and "wait_phase(&bars.empty" in tail and "rank" not in tail


def test_rows_are_released_and_acquired_at_cluster_scope():
    # the rows that one CTA's warps copied are read for the other CTA's thread
    import os
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                            "bit_weight_quantized_prepack_b200", "csrc", "wq_experts_large.cu")).read()
    gather = src[src.index("rows of the activations"):src.index("// ---------------------------------------------------------------- MMAs")]
    assert "mbar_arrive_leader_release(&bars.full" in gather and "mbar_arrive_leader(" not in gather
    mma = src[src.index("// ---------------------------------------------------------------- MMAs"):src.index("---- weights")]
    assert "wait_phase<true>(&bars.full" in mma
    assert "wait_phase(&bars.full" not in mma and "mbar_test_wait(&bars.full" not in mma
