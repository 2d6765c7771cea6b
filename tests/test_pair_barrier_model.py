"""How two warps that share rows of the paged attention leave when a wait gives up:
every order of their steps, on the CPU.

The two meet at a barrier without a limit (`bar.sync` of 64 threads) once per unit
and at two of them in a row per piece, and at other places either may stop alone: a
bounded wait runs out, or it is the first to see the CTA's stop. A warp that stops
marks its row maxima, sets the stop and arrives once at either barrier without
waiting; its partner looks for the mark or the stop behind the barriers. The model
takes these rules as they stand in attn_paged_kernel and looks for an order in which
a warp waits for ever."""
import pytest

# One warp's steps: two pieces of two units. 'wait': bounded, may run out, and ends at the stop; 'wait blind':
# the same, but does not look at the stop; 'vote': meets the partner at barrier 0, then looks for its mark;
# 'meet 0', 'meet 1': only meets.
UNIT = ["wait", "vote", "wait blind", "wait"]
EPILOGUE = ["meet 0", "meet 1", "wait"]
STEPS = (UNIT * 2 + EPILOGUE) * 2


def stuck_orders(arrives=(0, 1), looks=True):
    """States in which some warp can never go on. A warp: (step, state), state 'run',
    'at' (in a barrier), 'woken' or 'gone'; shared: arrivals at either barrier, the
    stop, the warps' marks. A warp that stops arrives at the barriers `arrives`."""
    start = ((0, "run"), (0, "run"), (0, 0), False, (False, False))
    seen, todo, stuck = {start}, [start], []
    bar_of = lambda at: int(STEPS[at] == "meet 1")  # noqa: E731
    while todo:
        now = todo.pop()
        nxt = []
        w, (counts, stop, marks) = now[:2], now[2:]

        def arrive(both, n, bar):
            """One more arrival at a barrier; the second opens it for whoever waits there."""
            n[bar] += 1
            if n[bar] == 2:
                n[bar] = 0
                for j in (0, 1):
                    if both[j][1] == "at" and bar_of(both[j][0]) == bar:
                        both[j] = (both[j][0], "woken")

        def put(i, me, bars=(), gives_up=False):
            both, n, m = list(w), list(counts), list(marks)
            both[i] = me
            for bar in bars:
                arrive(both, n, bar)
            m[i] = m[i] or gives_up
            nxt.append((*both, tuple(n), stop or gives_up, tuple(m)))

        if not stop:
            nxt.append((*w, counts, True, marks))      # another of the CTA's warps stops
        for i in (0, 1):
            at, state = w[i]
            leave = lambda: put(i, (at, "gone"), arrives, True)  # noqa: E731,B023
            if state in ("gone", "at"):
                continue
            if at == len(STEPS):
                put(i, (at, "gone"))
            elif state == "woken":                     # behind a barrier
                leave() if STEPS[at] == "vote" and marks[1 - i] and looks else put(i, (at + 1, "run"))
            elif STEPS[at].startswith("wait"):
                leave()                                # it ran out, or saw the stop
                if STEPS[at] == "wait blind" or not stop or not looks:
                    put(i, (at + 1, "run"))
            else:
                put(i, (at, "at"), (bar_of(at),))
        if stop and not nxt and any(x[1] == "at" for x in w):
            stuck.append(now)
        for s in nxt:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return stuck


def test_no_order_leaves_a_warp_at_a_barrier():
    assert not stuck_orders()


@pytest.mark.parametrize("arrives,looks", [((), True), ((0,), True), ((0, 1), False)])
def test_the_model_finds_orders_that_do(arrives, looks):
    assert stuck_orders(arrives, looks)
