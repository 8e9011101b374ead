"""The barrier protocols of the 8-bit products on the tensor cores (csrc/int8_mma.cu, int8_few.cu) as coroutines under random schedules.
A wait knows which phase it means and tests its parity alone, as the hardware does: run() raises Stuck where nobody can go on, or where a
wait takes another phase for its own."""


class Stuck(Exception):
    pass


class Barrier:
    def __init__(self, count):
        self.count = self.left = count
        self.phases = 0  # completed ones

    def arrive(self):
        assert self.left > 0
        self.left -= 1
        if self.left == 0:
            self.phases, self.left = self.phases + 1, self.count


def barriers(n, count):
    return [Barrier(count) for _ in range(n)]


def run(roles, rng):
    """roles: coroutines that yield None (go on), a list (wait until it has something) or (barrier, phase); phase -1: before the first."""
    waits = {i: next(r, "end") for i, r in enumerate(roles)}
    slow = []
    while True:
        waits = {i: w for i, w in waits.items() if w != "end"}
        if not waits:
            return
        if rng.random() < 0.01:  # some roles stand still for a while
            slow = rng.sample(range(len(roles)), rng.randint(0, 3))
        can = []
        for i, w in waits.items():
            if w is None or (isinstance(w, list) and w):
                can.append(i)
            elif isinstance(w, tuple) and (w[0].phases - 1) % 2 == w[1] % 2:
                if w[0].phases <= w[1]:
                    raise Stuck("role %d takes phase %d for phase %d" % (i, w[0].phases - 1, w[1]))
                can.append(i)
        if not can:
            raise Stuck("nobody can go on")
        fast = [i for i in can if i not in slow]
        i = rng.choice(fast if fast and rng.random() < 0.98 else can)
        waits[i] = next(roles[i], "end")


def arrivals(queue, n, rng=None):
    """The n arrivals that copies (in any order) or products (in theirs) make when they are done."""
    for _ in range(n):
        while not queue:
            yield queue
        queue.pop(rng.randrange(len(queue)) if rng else 0).arrive()
        yield None


def land(full, steps, places):
    """What a copier does when it has issued everything."""
    for i in range(max(0, steps - places), steps):
        yield full[i % places], i // places


def persistent(rng, parts, w_steps, x_steps, last_by_accumulators=False):
    """parts: the steps of each of a CTA's parts.  last_by_accumulators: the converting warps wait for the accumulators of the last part, and
    on the way for those of the part before the last one, instead of for all products."""
    w_full, w_empty = barriers(w_steps, 1), barriers(w_steps, 8)
    x_full, x_empty, ready = barriers(x_steps, 1), barriers(x_steps, 1), barriers(x_steps, 8)
    acc_full, acc_empty, done = barriers(2, 1), barriers(2, 4), Barrier(1)
    copies, products, last = [], [], len(parts) - 1

    def copier(full, empty, places):
        for i in range(sum(parts)):
            yield empty[i % places], i // places - 1
            copies.append(full[i % places])
            yield None
        yield from land(full, sum(parts), places)

    def multiplier():
        i = 0
        for t, n in enumerate(parts):
            yield acc_empty[t % 2], t // 2 - 1
            for _ in range(n):
                yield x_full[i % x_steps], i // x_steps
                yield ready[i % x_steps], i // x_steps
                products.append(x_empty[i % x_steps])
                yield None
                i += 1
            products.append(acc_full[t % 2])
        products.append(done)

    def finish():
        yield (acc_full[last % 2], last // 2) if last_by_accumulators else (done, 0)

    def converter(turn):
        i = 0
        for t, n in enumerate(parts):
            if last_by_accumulators and t >= 2:
                yield acc_full[t % 2], t // 2 - 1
            for _ in range(n):
                if i % 2 == turn:
                    yield w_full[i % w_steps], i // w_steps
                    if i >= 2:
                        yield x_empty[(i - 2) % x_steps], (i - 2) // x_steps
                    w_empty[i % w_steps].arrive()
                    ready[i % x_steps].arrive()
                    yield None
                i += 1
        yield from finish()

    def epilogue():
        for t in range(last):
            yield acc_full[t % 2], t // 2
            yield None
            acc_empty[t % 2].arrive()
        yield from finish()
    return [copier(w_full, w_empty, w_steps), copier(x_full, x_empty, x_steps), multiplier(), arrivals(copies, 2 * sum(parts), rng),
            arrivals(products, sum(parts) + len(parts) + 1)] + [converter(w // 8) for w in range(16)] + [epilogue() for _ in range(4)]


def cluster(rng, steps, places, waits_for_all=False):
    """A CTA's steps of a tile that a cluster shares.  waits_for_all: each converting warp waits for the copies of every step, not of its own."""
    full, ready, empty, done = barriers(places, 1), barriers(places, 8), barriers(places, 1), Barrier(1)
    copies, products = [], []

    def copier():
        for i in range(steps):
            if i >= places:
                yield empty[i % places], i // places - 1
            copies.append(full[i % places])
            yield None
        yield from land(full, steps, places)

    def multiplier():
        for i in range(steps):
            yield ready[i % places], i // places
            products.append(empty[i % places])
            yield None
        products.append(done)

    def converter(turn):
        for i in range(steps):
            if waits_for_all or i % 2 == turn:
                yield full[i % places], i // places
            if i % 2 == turn:
                if i >= 2:
                    yield empty[(i - 2) % places], (i - 2) // places
                ready[i % places].arrive()
                yield None
        yield done, 0
    return [copier(), multiplier(), arrivals(copies, steps, rng), arrivals(products, steps + 1)] + [converter(w // 8) for w in range(16)]
