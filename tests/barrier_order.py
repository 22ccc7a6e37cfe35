"""The order that barriers leave to the agents of a kernel: its roles' programs as a graph, and what of it is not safe.

An agent is a warp, a thread or an engine that works off what it is given in order.  A wait names a phase of an mbarrier
by its parity alone, so it is sound if the phase before is complete when the agent comes to it and the phase behind cannot
be before the agent has left; an arrival counts to the phase meant if that before is complete; two accesses of a place, one
of them a write, have to be in an order.  Each holds for every timing if it follows from the programs' order and the waits.
"""


class Order:
    def __init__(self):
        self.names, self.after, self.last = [], [], {}  # a node's name, the nodes it comes behind; an agent's last node
        self.count, self.arrivals, self.waits, self.accesses = {}, {}, [], {}

    def op(self, agent, name, after=()):
        self.names.append((agent, name))
        self.after.append([self.last[agent], *after] if agent in self.last else list(after))
        self.last[agent] = len(self.names) - 1
        return self.last[agent]

    def arrive(self, agent, bar, phase, count, after=()):
        """One of the `count` arrivals of a phase."""
        self.count[bar] = count
        self.arrivals.setdefault((bar, phase), []).append(self.op(agent, f"arrives at {bar} {phase}", after))

    def wait(self, agent, bar, phase):
        if phase >= 0:  # (the phase before the first is complete)
            self.waits.append((self.op(agent, f"waits for {bar} {phase}"), bar, phase))

    def touch(self, agent, kind, place, tag, after=()):
        """kind r, w or a (an addition: in any order with others of its tag); a read is to see what was written with its tag."""
        self.accesses.setdefault(place, []).append((self.op(agent, f"{kind} {place} {tag}", after), kind, tag))

    def faults(self):
        out = []
        for node, bar, phase in self.waits:
            got = self.arrivals.get((bar, phase), [])
            if len(got) != self.count[bar]:
                out.append(f"{self.names[node]}: {len(got)} arrivals")
        came = [list(x) for x in self.after]
        for node, bar, phase in self.waits:
            came[node] += self.arrivals[bar, phase]
        before, done = [0] * len(came), [0] * len(came)  # bits of the nodes that a node is behind
        for root in range(len(came)):
            stack = [root]
            while stack:
                n = stack[-1]
                left = [p for p in came[n] if done[p] != 2]
                if done[n] == 2:
                    stack.pop()
                elif left and done[n] == 1 and any(done[p] == 1 for p in left):
                    return out + [f"{self.names[n]}: waits for itself"]
                elif left:
                    done[n] = 1
                    stack += left
                else:
                    for p in came[n]:
                        before[n] |= before[p] | 1 << p
                    done[n] = 2
                    stack.pop()

        def first(x, y):
            return before[y] >> x & 1

        for node, bar, phase in self.waits:
            behind = self.arrivals.get((bar, phase + 1))
            if behind and not any(first(node, a) for a in behind):
                out.append(f"{self.names[node]}: the phase behind may be complete too")
            own = [p for p in self.after[node] if self.names[p][0] == self.names[node][0]]
            if any(not any(a == p or first(a, p) for p in own) for a in self.arrivals.get((bar, phase - 1), ())):
                out.append(f"{self.names[node]}: the phase before may not be complete")
        for (bar, phase), arrivals in self.arrivals.items():
            if any(not first(a, b) for a in self.arrivals.get((bar, phase - 1), ()) for b in arrivals):
                out.append(f"arrivals at {bar} {phase} may count to the phase before")
        for place, all_of in self.accesses.items():
            for i, (x, kind, tag) in enumerate(all_of):
                for y, kind2, tag2 in all_of[i + 1:]:
                    alike = kind == kind2 == "r" or (kind == kind2 == "a" and tag == tag2)
                    if not alike and not first(x, y) and not first(y, x):
                        out.append(f"{self.names[x]}, {self.names[y]}: in no order")
                if kind == "r":
                    wrote = [(y, k, t) for y, k, t in all_of if k != "r" and first(y, x)]
                    if any(k == "w" and t != tag and not any(first(y, z) and u == tag for z, _, u in wrote) for y, k, t in wrote):
                        out.append(f"{self.names[x]}: sees another's")
        return out
