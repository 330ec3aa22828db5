"""A model check, on the CPU, of the mbarrier protocol of the tree attention kernel: one CTA that runs
through a list of segments (pieces of one to several 128-key blocks).

Every role (the copying warp, two warps for masks, the MMA-issuing thread, four warps that take V,
queries and output, eight softmax warps) is an agent that issues, in the kernel's order, the same
waits and arrivals on the same barriers.  As for the prefill's model, a wait must name a phase that its
parity can tell, and every run has to end.  The rings' sizes are the kernel's; a ring of four descriptions,
with which the copying warp and the MMA thread wait for each other when segments are one block long, is
found to fail, and so are mask warps that do not wait for the queries' place."""
import random

import pytest

from barrier_model import Agent, Sim, Violation

ROW_RING, SC_RING = 4, 8


def tree_cta(rng, segs, fp8, blk, ring, seg_ring=8, masks_wait=True, rescale_p=0.03):
    """segs: [(blocks, first special block, active quads)]."""
    R = ring
    d = lambda lo, hi: ("delay", rng.uniform(lo, hi))
    first = [sum(s[0] for s in segs[:j]) for j in range(len(segs) + 1)]  # a segment's first block, running
    n_seg = len(segs)

    def bars(sim):
        for i in range(seg_ring):
            sim.bar(f"seg_full{i}", 1)
            sim.bar(f"seg_empty{i}", 15)
        for i in range(R):
            sim.bar(f"k_full{i}", 1)
            sim.bar(f"k_empty{i}", 1)
            sim.bar(f"v_full{i}", 1)
            sim.bar(f"v_empty{i}", 4 if fp8 else 1)
        for i in range(2):
            for name, c in (("s_full", 1), ("p_full", 12 if fp8 else 8), ("vt_empty", 1), ("q_ready", 6), ("q_free", 1),
                            ("tail_ready", 1), ("tail_done", 4)):
                sim.bar(f"{name}{i}", c)
        for i in range(SC_RING):
            sim.bar(f"sc_full{i}", 1)
            sim.bar(f"sc_empty{i}", 8)
        for i in range(ROW_RING):
            sim.bar(f"row_free{i}", 8)
        for i in range(4):
            sim.bar(f"meet{i}", 2)
        for name, c in (("o_full", 1), ("o_free", 4), ("drain", 1)):
            sim.bar(name, c)

    def seg_wait(j):
        return ("wait", f"seg_full{j % seg_ring}", j // seg_ring)

    def seg_give(j):
        return ("arrive", [f"seg_empty{j % seg_ring}"])

    def producer():
        made = 0
        batches = []  # (segment, block within it, blocks), fetched and not yet issued
        fj, fb, more = -1, 0, True
        g = 0
        while True:
            if more and (fj < 0 or fb == segs[fj][0]):
                fj += 1
                while made < min(fj + 2, n_seg + 1):
                    if made >= seg_ring:
                        yield ("wait", f"seg_empty{made % seg_ring}", made // seg_ring - 1)
                    yield ("arrive", [f"seg_full{made % seg_ring}"])
                    made += 1
                fb = 0
                more = fj < n_seg
            far = None
            if more:
                far = (fj, fb, min(4, segs[fj][0] - fb))
                fb += far[2]
            batches.append(far)
            if len(batches) == 3:
                cur = batches.pop(0)
                for _ in range(cur[2] if cur else 0):
                    if blk:
                        if g >= SC_RING:
                            yield ("wait", f"sc_empty{g % SC_RING}", g // SC_RING - 1)
                        yield ("arrive", [f"sc_full{g % SC_RING}"])
                    for x in "kv":
                        if g >= R:
                            yield ("wait", f"{x}_empty{g % R}", g // R - 1)
                        yield d(0.0, 0.2)
                        yield ("tma", f"{x}_full{g % R}")
                    g += 1
                if not more and not any(batches):
                    break
            elif not more and not any(batches):
                break
        for x in range(max(0, g - R), g):  # no copy in flight at the end
            yield ("wait", f"k_full{x % R}", x // R)
            yield ("wait", f"v_full{x % R}", x // R)

    def masks():
        for j in range(n_seg + 1):
            yield seg_wait(j)
            yield seg_give(j)
            if j == n_seg:
                break
            if j >= 2 and masks_wait:
                yield ("wait", f"q_free{j % 2}", j // 2 - 1)
            if j >= ROW_RING:
                yield ("wait", f"row_free{j % ROW_RING}", j // ROW_RING - 1)
            yield d(0.0, 2.0)
            yield ("arrive", [f"q_ready{j % 2}"])

    def special(j, b):
        return b >= segs[j][1]

    def mma():
        total = first[n_seg]
        gq, jq, bq, tq = 0, -1, 0, 0
        gp, jp, bp, tp = 0, -1, 0, 0
        q_end = False
        lead = 0
        while True:
            if lead >= 2:
                if jp < 0 or bp == segs[jp][0]:
                    jp += 1
                    yield seg_wait(jp)
                    yield seg_give(jp)
                    if jp == n_seg:
                        break
                    bp = 0
                    if jp > 0:
                        yield ("wait", "o_free", jp - 1)
                yield ("wait", f"p_full{gp % 2}", gp // 2)
                if not fp8:
                    yield ("wait", f"v_full{gp % R}", gp // R)
                    if special(jp, bp):
                        yield ("wait", f"tail_done{tp % 2}", tp // 2)
                        tp += 1
                yield d(0.0, 0.5)
                bp += 1
                yield ("mma", [f"vt_empty{gp % 2}" if fp8 else f"v_empty{gp % R}"] + (["o_full"] if bp == segs[jp][0] else []))
                gp += 1
            lead += 1
            if not q_end and (jq < 0 or bq == segs[jq][0]):
                jq += 1
                yield seg_wait(jq)
                if jq == n_seg:
                    q_end = True
                else:
                    bq = 0
                    yield ("wait", f"q_ready{jq % 2}", jq // 2)
            if not q_end:
                yield ("wait", f"k_full{gq % R}", gq // R)
                if not fp8 and special(jq, bq):
                    yield ("arrive", [f"tail_ready{tq % 2}"])
                    tq += 1
                yield d(0.0, 0.5)
                bq += 1
                yield ("mma", [f"s_full{gq % 2}", f"k_empty{gq % R}"] + ([f"q_free{jq % 2}"] if bq == segs[jq][0] else []))
                gq += 1
        assert gp == total == gq
        yield ("mma", ["drain"])
        yield ("wait", "drain", 0)

    def values():
        g = t = 0

        def store(j):
            if j >= 2:
                yield ("wait", f"q_free{j % 2}", j // 2 - 1)
            if j >= ROW_RING:
                yield ("wait", f"row_free{j % ROW_RING}", j // ROW_RING - 1)
            yield d(0.1, 1.0)
            yield ("arrive", [f"q_ready{j % 2}"])

        def write(j):
            yield ("wait", f"row_free{j % ROW_RING}", j // ROW_RING)
            yield ("wait", "o_full", j)
            yield d(0.1, 1.5)
            yield ("arrive", ["o_free"])

        for j in range(-1, n_seg + 1):
            end = j == n_seg
            n = 0 if j < 0 or end else segs[j][0]
            ahead = False
            if not end:
                yield seg_wait(j + 1)
                ahead = j + 1 < n_seg
            b = 0
            while True:
                if b < n:
                    if fp8:
                        yield ("wait", f"v_full{g % R}", g // R)
                        if g >= 2:
                            yield ("wait", f"vt_empty{g % 2}", g // 2 - 1)
                        yield d(0.2, 1.0)
                        yield ("arrive", [f"p_full{g % 2}", f"v_empty{g % R}"])
                    elif special(j, b):
                        yield ("wait", f"tail_ready{t % 2}", t // 2)
                        yield ("wait", f"v_full{g % R}", g // R)
                        yield d(0.0, 0.5)
                        yield ("arrive", [f"tail_done{t % 2}"])
                        t += 1
                    g += 1
                if ahead and b == (0 if n < 4 else 3):
                    yield from store(j + 1)
                if b == 0 and j > 0:
                    yield from write(j - 1)
                    yield seg_give(j - 1)
                b += 1
                if b >= n:
                    break

    def softmax(quad):
        g = xk = 0
        for j in range(n_seg + 1):
            yield seg_wait(j)
            yield seg_give(j)
            if j == n_seg:
                break
            active = quad >= 4 - segs[j][2]
            for b in range(segs[j][0]):
                if blk:
                    yield ("wait", f"sc_full{g % SC_RING}", g // SC_RING)
                yield ("wait", f"s_full{g % 2}", g // 2)
                if active:
                    yield d(0.1, 0.6)
                    yield ("arrive", [f"meet{quad}"])
                    yield ("wait", f"meet{quad}", xk)
                    xk += 1
                    if b > 0 and rng.random() < rescale_p:
                        yield ("wait", f"vt_empty{(g - 1) % 2}", (g - 1) // 2) if fp8 else ("wait", f"v_empty{(g - 1) % R}", (g - 1) // R)
                    yield d(0.3, 1.0)
                yield ("arrive", ([f"sc_empty{g % SC_RING}"] if blk else []) + [f"p_full{g % 2}"])
                g += 1
            yield ("arrive", [f"row_free{j % ROW_RING}"])
        yield ("arrive", [f"meet{quad}"])  # the last meeting
        yield ("wait", f"meet{quad}", xk)

    agents = [Agent("producer", producer()), Agent("mma", mma())]
    agents += [Agent(f"mask{i}", masks()) for i in range(2)]
    agents += [Agent(f"values{i}", values()) for i in range(4)]
    agents += [Agent(f"softmax{i}", softmax(i % 4)) for i in range(8)]
    return bars, agents


def run_once(seed, fp8, blk, ring, longest, **kw):
    rng = random.Random(seed)
    segs = []
    for _ in range(rng.choice([0, 1, 2, 3, 6, 12])):
        n = rng.randint(1, longest)
        segs.append((n, rng.randint(max(0, n - 3), n), rng.randint(1, 4)))
    sim = Sim(rng, 25.0)
    bars, agents = tree_cta(rng, segs, fp8, blk, ring, **kw)
    bars(sim)
    sim.run(agents)


@pytest.mark.parametrize("fp8,blk,ring", [(True, False, 3), (True, True, 3), (False, False, 3), (False, False, 4)])
@pytest.mark.parametrize("longest", [1, 2, 5, 11])
def test_kernel_protocol_holds_on_random_schedules(fp8, blk, ring, longest):
    for seed in range(250):
        run_once(seed * 7 + longest, fp8, blk, ring, longest)


@pytest.mark.parametrize("kw", [dict(seg_ring=4), dict(masks_wait=False)])
def test_faulty_protocols_are_caught(kw):
    found = 0
    for seed in range(200):
        try:
            run_once(seed, False, False, 3, 1, **kw)
        except Violation:
            found += 1
    assert found > 0
