"""A randomised model of the barrier protocol of the windowed and tree decodes'
tensor-core kernel (`mla_decode_context_gb300/csrc/dcp_decode_select.cu`), built
on the machinery of `decode_protocol_model`: the same barriers, arrival counts,
parities and ring sizes, role by role, run under random interleavings with
every asynchronous completion delivered at a random later time.

A cluster walks a list of units of `sizes` tiles each.  The score CTA's stage
ring carries items: four of a unit's Q, then its tiles.  Checked as in the
plain decode's model (deadlock, over-arrival, phases that mix tiles, aliased
parity waits, buffers overwritten or read too early), and besides:
  * Q in TMEM is not overwritten while an MMA of the previous unit reads it,
    nor read before all four quarters are there;
  * O is not overwritten by a unit's first PV before the previous unit's
    epilogue has read it, and an epilogue sees exactly its unit's PVs;
  * a unit's 1/l is read before its slot takes a later unit's, and the two
    softmax groups' sums meet unit by unit;
  * a descriptor is not rewritten while a role still uses it.
"""
from __future__ import annotations

from tests import decode_protocol_model as P

ProtocolError = P.ProtocolError
K_Q, K_UNITS, K_FIN = 4, 3, 8
PTX = 128 * 32 * 2 + 4 * 144
HALF = P.HALF
ST, OWN, RECV, PS = P.K_STAGES, P.K_OWN, P.K_RECV, P.K_PSLOTS
SB = 4                               # S slots, one issuing warp each
DONE = set(range(P.K_SPARTS))        # what the plain decode's model calls a finished S


class Model(P.Model):
    def __init__(self, sizes, seed, mutation=None, decoupled=True, rescale_prob=0.3):
        self.sizes = list(sizes)
        self.j0 = [sum(self.sizes[:k]) for k in range(len(self.sizes) + 1)]
        self.g0 = [self.j0[k] + K_Q * k for k in range(len(self.sizes) + 1)]
        super().__init__(self.j0[-1], seed, rescale_prob=rescale_prob, mutation=mutation, decoupled=decoupled)
        self.seen = [0] * SB
        self.sslot = [dict(tile=None, parts_done=0, read=True) for _ in range(SB)]
        self.q_tmem = [None] * K_Q       # the unit whose quarter is in TMEM
        self.s_running = 0               # tiles whose S is issued and not complete
        self.o_unit, self.o_pvs, self.o_read = None, set(), True
        self.fin_slot = [None] * K_FIN
        self.fin_sh = [dict(unit=None, groups=set(), read=True) for _ in range(2)]
        self.desc = [dict(unit=None, users=0) for _ in range(K_UNITS)]

    def _mk_barriers(self):
        def mk(cta, name, n, count):
            for i in range(n):
                self.bars[(cta, name, i)] = P.Bar("%s[%d]@%d" % (name, i, cta), count)
        # roles per CTA that use a descriptor, counted as the kernel counts warps
        self.users = {0: 2 + 1 + SB + 2, 1: (3 if self.decoupled else 2) + (0 if self.decoupled else 1) + 1 + 1 + 1 + 1}
        for cta in (0, 1):
            mk(cta, "kv_loaded", ST, 128)
            mk(cta, "kv_full", ST, 5)
            mk(cta, "s_done", ST, 1 if self.decoupled else 2)
            mk(cta, "own_loaded", OWN, 128)
            mk(cta, "own_free", OWN, 1)
            mk(cta, "q_gone", 1, 4)
            mk(cta, "v_full", RECV, 128 if self.decoupled else 1)
            mk(cta, "v_free", RECV, 1)
            mk(cta, "s_full", SB, 2)
            mk(cta, "s_free", SB, 4)
            mk(cta, "q_ready", 1, 4)
            mk(cta, "s_end", 1, SB)
            mk(cta, "p_full", PS, 1)
            mk(cta, "p_free", PS, 1)
            mk(cta, "p_ok", PS, 5)
            mk(cta, "pv_done", PS, 1)
            mk(cta, "o_final", 1, 1)
            mk(cta, "o_free", 1, 2)          # two epilogue halves (the kernel: 8 warps)
            mk(cta, "fin_l", K_FIN, 1)
            mk(cta, "m_pub", 2, 4)
            mk(cta, "sm_fin", 1, 2)          # two groups (the kernel: 8 warps)
            mk(cta, "ud_full", K_UNITS, 1)
            mk(cta, "ud_free", K_UNITS, self.users[cta])
        for i in range(PS):
            self.b(1, "p_full", i).txop(PTX)
            self.b(1, "p_full", i).arrive()
        if not self.decoupled:
            for i in range(RECV):
                self.b(1, "v_full", i).txop(HALF)
                self.b(1, "v_full", i).arrive()
        for i in range(K_FIN):
            self.b(1, "fin_l", i).txop(512)
            self.b(1, "fin_l", i).arrive()

    # ---------------------------------------------------------- descriptors
    def scheduler(self, cta):
        for k in range(len(self.sizes)):
            s = k % K_UNITS
            if self.mut != "scheduler_skips_free":
                yield self.W(cta, "ud_free", s, k // K_UNITS - 1)

            def put(k=k, s=s):
                d = self.desc_of(cta)[s]
                self.check(d["users"] == 0, "descriptor %s of unit %s rewritten (unit %s) in use", s, d["unit"], k)
                self.desc_of(cta)[s] = dict(unit=k, users=self.users[cta])
                self.b(cta, "ud_full", s).arrive(tag=k)
            yield ("do", put)

    def desc_of(self, cta):
        if not hasattr(self, "_desc"):
            self._desc = {c: [dict(unit=None, users=0) for _ in range(K_UNITS)] for c in (0, 1)}
        return self._desc[cta]

    def enter(self, cta, k):
        return self.W(cta, "ud_full", k % K_UNITS, k // K_UNITS)

    def leave(self, cta, k):
        def f():
            d = self.desc_of(cta)[k % K_UNITS]
            self.check(d["unit"] == k, "unit %s's descriptor is gone (slot holds %s)", k, d["unit"])
            d["users"] -= 1
            self.b(cta, "ud_free", k % K_UNITS).arrive(tag=k)
        return ("do", f)

    def item(self, g):
        """(unit, tile or None, quarter or None) of stage item g"""
        k = max(i for i in range(len(self.sizes)) if self.g0[i] <= g)
        n = g - self.g0[k]
        return (k, None, n) if n < K_Q else (k, self.j0[k] + n - K_Q, None)

    # ----------------------------------------------------------------- roles
    def score_producers(self, grp):
        for k in range(len(self.sizes)):
            yield self.enter(0, k)
            for g in range(self.g0[k], self.g0[k + 1]):
                if g % 2 != grp:
                    continue
                st = g % ST
                _, j, _ = self.item(g)
                if g >= ST and self.mut != "producers_uncoupled":
                    need = ((g - ST) >> 1) + 1
                    yield ("cond", lambda need=need: self.claimed[1 - grp] >= need)
                if self.mut != "producers_skip_stage_free":
                    yield self.W(0, "s_done", st, g // ST - 1)

                def claim(g=g):
                    self.claimed[grp] = max(self.claimed[grp], (g >> 1) + 1)
                yield ("do", claim)

                def write(g=g, st=st, j=j):
                    if self.stage[st]["tile"] != g:
                        self.claim_stage(st, g, "score producers")
                    if j is None:
                        self.stage[st]["cp_read"] = True
                    else:
                        m = self.mask[j % 16]
                        self.check(m["read"], "mask slot %s overwritten before tile %s's softmax", j % 16, m["tile"])
                        self.mask[j % 16] = dict(tile=j, read=False)
                yield ("do", write)
                if self.decoupled or j is None:
                    yield ("do", lambda st=st, g=g: self.b(0, "kv_full", st).arrive(tag=g))
                else:
                    yield ("do", lambda st=st, g=g: (self.b(0, "kv_full", st).txop(HALF),
                                                     self.b(0, "kv_full", st).arrive(tag=g)))
                for _ in range(3):
                    yield ("do", lambda st=st, g=g: self.b(0, "kv_full", st).arrive(tag=g))

                def landed(st=st, j=j):
                    self.stage[st]["own"] = True
                    if self.decoupled or j is None:
                        self.stage[st]["fwd"] = True
                    self.b(0, "kv_loaded", st).arrive(128)
                yield ("do", lambda f=landed: self.later(f))
            yield self.leave(0, k)

    def _units(self, cta, inner):
        for k in range(len(self.sizes)):
            yield self.enter(cta, k)
            yield from inner(k)
            yield self.leave(cta, k)

    def value_producers(self, grp):
        def inner(k):
            for j in range(self.j0[k], self.j0[k + 1]):
                if j % 2 != grp:
                    continue
                os_ = j % OWN
                yield self.W(1, "own_free", os_, j // OWN - 1)

                def write(j=j, os_=os_):
                    o = self.own[os_]
                    self.check(o["fwd_read"] and o["pv_read"], "own slot %s overwritten (tile %s) while tile %s still needed",
                               os_, j, o["tile"])
                    self.own[os_] = dict(tile=j, landed=False, fwd_read=self.decoupled, pv_read=False, fenced=False)
                yield ("do", write)

                def landed(os_=os_):
                    self.own[os_]["landed"] = True
                    self.b(1, "own_loaded", os_).arrive(128)
                yield ("do", lambda f=landed: self.later(f))
        yield from self._units(1, inner)

    def value_recv_producers(self):
        def inner(k):
            for j in range(self.j0[k], self.j0[k + 1]):
                vs = j % RECV
                yield self.W(1, "v_free", vs, j // RECV - 1)

                def write(j=j, vs=vs):
                    r = self.recv[vs]
                    self.check(r["pv_read"], "receive slot %s overwritten (tile %s) before PV(%s)", vs, j, r["tile"])
                    self.recv[vs] = dict(tile=j, landed=False, pv_read=False, fenced=False)
                yield ("do", write)

                def landed(vs=vs):
                    self.recv[vs]["landed"] = True
                    self.b(1, "v_full", vs).arrive(128)
                yield ("do", lambda f=landed: self.later(f))
        yield from self._units(1, inner)

    def score_forwarder(self):
        state = dict(gf=0, gc=0, jc=0)

        def inner(k):
            end = self.g0[k + 1]
            while state["gc"] < end:
                moved = False
                gf = state["gf"]
                if self.decoupled:
                    yield self.W(0, "kv_loaded", gf % ST, gf // ST)
                if gf < end and self.passed(0, "kv_loaded", gf % ST, gf // ST, "score fwd"):
                    st = gf % ST
                    self.check(self.stage[st]["tile"] == gf and self.stage[st]["own"],
                               "forwarder fenced stage %s for item %s before its rows landed", st, gf)
                    yield ("do", lambda st=st, gf=gf: self.b(0, "kv_full", st).arrive(tag=gf))
                    state["gf"] = gf + 1
                    moved = True
                if self.decoupled:
                    state["gc"] = state["gf"]
                elif state["gc"] < state["gf"]:
                    gc, jc = state["gc"], state["jc"]
                    if gc - self.g0[k] < K_Q:
                        state["gc"] = gc + 1
                        moved = True
                    elif self.passed(0, "v_free", jc % RECV, jc // RECV - 1, "score fwd"):
                        st, rs = gc % ST, jc % RECV

                        def copy(st=st, rs=rs, j=jc, g=gc):
                            r = self.recv[rs]
                            self.check(r["pv_read"], "receive slot %s overwritten (tile %s) before PV(%s)", rs, j, r["tile"])
                            self.check(self.stage[st]["tile"] == g, "copy of item %s from a stage holding %s", g, self.stage[st]["tile"])
                            self.recv[rs] = dict(tile=j, landed=False, pv_read=False, fenced=True)

                            def land():
                                self.stage[st]["cp_read"] = True
                                self.recv[rs]["landed"] = True
                                self.b(1, "v_full", rs).txop(-HALF)
                            self.later(land)
                        yield ("do", copy)
                        state["gc"], state["jc"] = gc + 1, jc + 1
                        moved = True
                if not moved:
                    yield ("yield",)
        yield from self._units(0, inner)

    def value_forwarder(self):
        state = dict(wg=0, turns=[0] * ST)

        def inner(k):
            for g in range(self.g0[k] + K_Q, self.g0[k + 1]):
                _, j, _ = self.item(g)
                st, n = g % ST, g - self.g0[k] - K_Q
                yield self.W(1, "own_loaded", j % OWN, j // OWN)
                if (n == 1 or self.sizes[k] == 1) and self.mut != "value_forwarder_skips_q":
                    yield self.W(1, "q_gone", 0, k)
                while state["wg"] <= g - ST:
                    if self.item(state["wg"])[1] is not None:
                        ws = state["wg"] % ST
                        yield self.W(1, "s_done", ws, state["turns"][ws])
                        state["turns"][ws] += 1
                    state["wg"] += 1

                def copy(g=g, j=j, st=st):
                    o = self.own[j % OWN]
                    self.check(o["tile"] == j and o["landed"], "value forwarder copies own slot before tile %s landed", j)

                    def land():
                        o["fwd_read"] = True
                        if self.stage[st]["tile"] != g:
                            self.claim_stage(st, g, "the value CTA's copy")
                        self.stage[st]["fwd"] = True
                        self.b(0, "kv_full", st).txop(-HALF)
                    self.later(land)
                yield ("do", copy)
        yield from self._units(1, inner)

    def recv_warp(self):
        def inner(k):
            for j in range(self.j0[k], self.j0[k + 1]):
                g = self.g0[k] + K_Q + j - self.j0[k]
                st, vs, os_ = g % ST, j % RECV, j % OWN
                yield self.W(1, "v_full", vs, j // RECV)

                def arrivals(st=st, vs=vs, g=g):
                    self.b(1, "v_full", vs).txop(HALF)
                    self.b(1, "v_full", vs).arrive()
                    self.b(1, "s_done", st).arrive(tag=g)
                    self.later(lambda: self.b(0, "s_done", st).arrive(tag=g))
                if not self.decoupled:
                    yield ("do", arrivals)
                yield self.W(1, "own_loaded", os_, j // OWN)

                def fence(j=j, os_=os_, vs=vs):
                    if self.own[os_]["tile"] == j and self.own[os_]["landed"]:
                        self.own[os_]["fenced"] = True
                    r = self.recv[vs]
                    if self.decoupled and r["tile"] == j and r["landed"]:
                        r["fenced"] = True
                yield ("do", fence)
                yield ("do", lambda j=j: self.b(1, "p_ok", j % PS).arrive(tag=j))
        yield from self._units(1, inner)

    def s_issuer(self, b):
        def inner(k):
            j0 = self.j0[k]
            if k > 0 and self.mut == "q_waits_for_s_full":
                for p in range(1, SB + 1):
                    if j0 >= p:
                        yield self.W(0, "s_full", (j0 - p) % SB, (j0 - p) // SB)
            elif k > 0 and self.mut != "q_over_running_s":
                yield self.W(0, "s_end", 0, k - 1)
            g = self.g0[k] + b
            st = g % ST
            yield self.W(0, "kv_full", st, g // ST)

            def move(st=st, g=g):
                s = self.stage[st]
                self.check(s["tile"] == g and s["own"], "Q quarter of item %s read from a stage holding %s", g, s["tile"])
                self.check(self.s_running == 0, "Q of unit %s overwrites TMEM while S runs", k)
                self.q_tmem[b] = k
                s["s_done"] = DONE
                n = 1 if self.decoupled else 2
                self.b(0, "s_done", st).arrive(n, tag=g)
            yield ("do", move)
            yield ("do", lambda: self.b(0, "q_ready", 0).arrive(tag=k))
            if not self.decoupled:
                yield ("do", lambda: self.later(lambda: self.b(1, "q_gone", 0).arrive(tag=k)))
            yield self.W(0, "q_ready", 0, k)
            for j in range(j0, self.j0[k + 1]):
                if j % SB != b:
                    continue
                g = self.g0[k] + K_Q + j - j0
                st = g % ST
                yield self.W(0, "s_free", b, j // SB - 1)
                if not self.decoupled and self.mut != "issuers_uncoupled":
                    yield ("cond", lambda j=j: self.seen[(j - ST) % SB] >= j - ST + 1)
                yield self.W(0, "kv_full", st, g // ST)

                def saw(j=j):
                    self.seen[b] = j + 1
                yield ("do", saw)

                def issue(j=j, g=g, st=st):
                    s = self.stage[st]
                    self.check(s["tile"] == g and s["own"] and s["fwd"], "S(%s) issued on stage %s holding item %s", j, st, s["tile"])
                    self.check(all(q == k for q in self.q_tmem), "S(%s) of unit %s issued with Q of %s", j, k, self.q_tmem)
                    sl = self.sslot[b]
                    if sl["tile"] != j:
                        self.check(sl["read"], "S slot %s rewritten (tile %s) before the softmax read tile %s", b, j, sl["tile"])
                        self.sslot[b] = dict(tile=j, parts_done=0, read=False)
                    self.b(0, "s_full", b).arrive(tag=j)
                    self.s_running += 1

                    def done():
                        self.s_running -= 1
                        self.sslot[b]["parts_done"] += 1
                        self.stage[st]["s_done"] = DONE
                        self.b(0, "s_full", b).arrive(tag=j)
                        self.b(0, "s_done", st).arrive(tag=g)
                        if not self.decoupled:
                            self.b(1, "s_done", st).arrive(tag=g)
                    self.later(done, fifo=("S", b))
                yield ("do", issue)
            yield ("do", lambda: self.later(lambda: self.b(0, "s_end", 0).arrive(tag=k), fifo=("S", b)))
        yield from self._units(0, inner)

    def softmax(self, grp):
        def inner(k):
            j0 = self.j0[k]
            for j in range(j0, self.j0[k + 1]):
                if j % 2 != grp:
                    continue
                b, slot, i = j % SB, j % PS, j - j0
                if i == 1:
                    yield self.W(0, "m_pub", k % 2, k // 2)

                    def read_m(j=j):
                        m = self.mring[k % 2]
                        self.check(m["tile"] == j - 1, "tile %s read tile %s's max", j, m["tile"])
                        m["reads_left"] -= 1
                    yield ("do", read_m)
                yield self.W(0, "s_full", b, j // SB)

                def read_s(j=j, b=b):
                    sl = self.sslot[b]
                    self.check(sl["tile"] == j and sl["parts_done"] == 1, "softmax read S slot %s for tile %s: holds %s (%s parts)",
                               b, j, sl["tile"], sl["parts_done"])
                    m = self.mask[j % 16]
                    self.check(m["tile"] == j, "mask slot %s holds tile %s, wanted %s", j % 16, m["tile"], j)
                    m["read"] = True
                    sl["read"] = True
                yield ("do", read_s)
                for _ in range(4):
                    yield ("do", lambda b=b, j=j: self.b(0, "s_free", b).arrive(tag=j))

                if i == 0:
                    def post(j=j):
                        m = self.mring[k % 2]
                        self.check(m["reads_left"] <= 0, "unit %s's first max overwritten by tile %s unread", k - 2, j)
                        self.mring[k % 2] = dict(tile=j, reads_left=1 if self.sizes[k] > 1 else 0)
                    yield ("do", post)
                    for _ in range(4):
                        yield ("do", lambda j=j: self.b(0, "m_pub", k % 2).arrive(tag=j))
                yield self.W(0, "p_free", slot, j // PS - 1)

                def send(j=j, slot=slot):
                    self.check(self.stg[slot]["reads_left"] == 0, "P staging slot %s rewritten (tile %s) before its copies read it", slot, j)
                    p = self.pslot[slot]
                    self.check(p["pv_read"] and p["max_read"], "P slot %s refilled (tile %s) before tile %s was consumed", slot, j, p["tile"])
                    self.stg[slot] = dict(tile=j, reads_left=8)
                    self.pslot[slot] = dict(tile=j, bytes=0, pv_read=False, max_read=False)
                    for _ in range(8):
                        def land(slot=slot):
                            self.stg[slot]["reads_left"] -= 1
                            self.pslot[slot]["bytes"] += PTX // 8
                            self.b(1, "p_full", slot).txop(-(PTX // 8))
                        self.later(land)
                yield ("do", send)
            if k > 0 and self.mut != "sm_fin_without_wait":
                yield self.W(0, "sm_fin", 0, k - 1)

            def put():
                f = self.fin_sh[k & 1]
                if f["unit"] != k:
                    self.check(f["read"], "sums of unit %s overwritten (unit %s) unread", f["unit"], k)
                    self.fin_sh[k & 1] = dict(unit=k, groups=set(), read=False)
                self.fin_sh[k & 1]["groups"].add(grp)
                self.b(0, "sm_fin", 0).arrive(tag=k)
            yield ("do", put)
            if grp == 0:
                yield self.W(0, "sm_fin", 0, k)

                def finish():
                    f = self.fin_sh[k & 1]
                    self.check(f["unit"] == k and f["groups"] == {0, 1}, "unit %s finished with sums of %s (%s)", k, f["unit"], f["groups"])
                    f["read"] = True

                    def land():
                        s = self.fin_slot[k % self.nfin]
                        self.check(s is None, "1/l of unit %s overwritten (unit %s)", s, k)
                        self.fin_slot[k % self.nfin] = k
                        self.b(1, "fin_l", k % self.nfin).txop(-512)
                    self.later(land)
                yield ("do", finish)
        yield from self._units(0, inner)

    @property
    def nfin(self):
        return 2 if self.mut == "two_fin_slots" else K_FIN

    def value_max_and_epilogue(self, half):
        """warps 0-3 (half 0: max tracking, then their epilogue columns) or
        warps 4-7 (half 1: epilogue only)"""
        def inner(k):
            j0, j1 = self.j0[k], self.j0[k + 1]
            if half == 0:
                for j in range(j0, j1):
                    slot = j % PS
                    yield self.W(1, "p_full", slot, j // PS)

                    def rearm(slot=slot, j=j):
                        p = self.pslot[slot]
                        self.check(p["tile"] == j and p["bytes"] == PTX // 8 * 8, "P(%s) seen incomplete in slot %s", j, slot)
                        p["max_read"] = True
                        self.b(1, "p_full", slot).txop(PTX // 8 * 8)
                        self.b(1, "p_full", slot).arrive()
                    yield ("do", rearm)
                    if self.rng.random() < 0.1:      # clearing non-finite values
                        yield self.W(1, "v_full", j % RECV, j // RECV)
                        yield self.W(1, "own_loaded", j % OWN, j // OWN)
                        yield ("do", lambda j=j: self.check(self.own[j % OWN]["tile"] == j and self.recv[j % RECV]["tile"] == j,
                                                            "V(%s) cleared in slots holding other tiles", j))
                    if j > j0 and self.rng.random() < self.rescale_prob:
                        yield self.W(1, "pv_done", (j - 1) % PS, (j - 1) // PS)
                        yield ("do", lambda j=j: self.check(self.o_unit == k and j - 1 in self.o_pvs, "O rescaled before PV(%s)", j - 1))
                    for _ in range(4):
                        yield ("do", lambda slot=slot, j=j: self.b(1, "p_ok", slot).arrive(tag=j))
            if self.mut == "epilogue_waits_for_pv_done":
                yield self.W(1, "pv_done", (j1 - 1) % PS, (j1 - 1) // PS)
            else:
                yield self.W(1, "o_final", 0, k)
            f = k % self.nfin
            yield self.W(1, "fin_l", f, k // self.nfin)

            def read():
                self.check(self.o_unit == k and self.o_pvs == set(range(j0, j1)), "epilogue of unit %s on O of unit %s with %s",
                           k, self.o_unit, sorted(self.o_pvs))
                self.check(self.fin_slot[f] == k, "1/l of unit %s read as unit %s's", self.fin_slot[f], k)
                self.epi_done.setdefault(k, set()).add(half)
                self.b(1, "o_free", 0).arrive(tag=k)
                if half == 0:
                    self.rearmed = k
            yield ("do", read)
            if half == 0:
                def rearm_fin():
                    self.b(1, "fin_l", f).txop(512)
                    self.b(1, "fin_l", f).arrive()
                    self.fin_cleared(k)
                yield ("do", rearm_fin)
            else:
                yield ("do", lambda: self.fin_cleared(k))
        yield from self._units(1, inner)

    def fin_cleared(self, k):
        c = self.fin_seen.setdefault(k, 0) + 1
        self.fin_seen[k] = c
        if c == 2 and self.fin_slot[k % self.nfin] == k:
            self.fin_slot[k % self.nfin] = None

    def pv_issuer(self):
        def inner(k):
            if k > 0 and self.mut != "pv_over_unread_o":
                yield self.W(1, "o_free", 0, k - 1)
            for j in range(self.j0[k], self.j0[k + 1]):
                vs, os_, slot = j % RECV, j % OWN, j % PS
                yield self.W(1, "p_ok", slot, j // PS)

                def issue(j=j, vs=vs, os_=os_, slot=slot):
                    self.check(self.pslot[slot]["tile"] == j and self.pslot[slot]["bytes"] == PTX // 8 * 8, "PV(%s) issued before P landed", j)
                    self.check(self.recv[vs]["tile"] == j and self.recv[vs]["landed"] and self.recv[vs]["fenced"], "PV(%s) issued before chunks 0-3", j)
                    self.check(self.own[os_]["tile"] == j and self.own[os_]["landed"] and self.own[os_]["fenced"], "PV(%s) issued before chunks 4-7", j)
                    if j == self.j0[k]:
                        if k > 0:
                            self.check(self.epi_done.get(k - 1, set()) == {0, 1}, "unit %s overwrites O before unit %s's was read", k, k - 1)
                        self.o_unit, self.o_pvs = k, set()

                    def done():
                        self.recv[vs]["pv_read"] = True
                        self.own[os_]["pv_read"] = True
                        self.pslot[slot]["pv_read"] = True
                        self.o_pvs.add(j)
                        self.b(0, "v_free", vs).arrive()
                        self.b(1, "v_free", vs).arrive()
                        self.b(1, "own_free", os_).arrive()
                        self.b(0, "p_free", slot).arrive()
                        self.b(1, "p_free", slot).arrive()
                        self.b(1, "pv_done", slot).arrive()
                        if j == self.j0[k + 1] - 1:
                            self.b(1, "o_final", 0).arrive(tag=k)
                    self.later(done, fifo=("PV",))
                yield ("do", issue)
        yield from self._units(1, inner)

    def roles(self):
        self.epi_done, self.fin_seen = {}, {}
        r = {"sched0": self.scheduler(0), "sched1": self.scheduler(1), "fwd0": self.score_forwarder(),
             "recv": self.recv_warp(), "vmax": self.value_max_and_epilogue(0), "epi": self.value_max_and_epilogue(1),
             "pv": self.pv_issuer()}
        if self.decoupled:
            r["vp2"] = self.value_recv_producers()
        else:
            r["fwd1"] = self.value_forwarder()
        for g in (0, 1):
            r["sp%d" % g] = self.score_producers(g)
            r["vp%d" % g] = self.value_producers(g)
            r["sm%d" % g] = self.softmax(g)
        for b in range(SB):
            r["s%d" % b] = self.s_issuer(b)
        # every role uses each descriptor of its CTA once
        n0 = sum(x.startswith(("sp", "sm", "s0", "s1", "s2", "s3", "fwd0")) for x in r)
        n1 = len(r) - 2 - n0
        assert (n0, n1) == (self.users[0], self.users[1]), (n0, n1, self.users)
        return r

    def run(self):
        roles = self.roles()
        cur = {name: None for name in roles}
        finished = set()
        steps = idle_polls = 0
        while True:
            steps += 1
            if steps > 3_000_000:
                raise ProtocolError("no progress")
            runnable = []
            for name, gen in roles.items():
                if name in finished:
                    continue
                if cur[name] is None:
                    try:
                        cur[name] = next(gen)
                    except StopIteration:
                        finished.add(name)
                        continue
                op = cur[name]
                if op[0] == "cond":
                    if op[1]():
                        runnable.append(name)
                elif op[0] == "wait":
                    _, cta, bname, i, t = op
                    bar = self.b(cta, bname, i)
                    if (bar.done & 1) != (t & 1):
                        if bar.done != t + 1:
                            raise ProtocolError("aliased wait on %s by %s: %d phases done, target phase %d"
                                                % (bar.name, name, bar.done, t))
                        runnable.append(name)
                    elif bar.done > t + 1:
                        raise ProtocolError("%s waits on %s for phase %d, already %d done" % (name, bar.name, t, bar.done))
                else:
                    runnable.append(name)
            busy = [n for n in runnable if cur[n][0] != "yield"]
            polling = [n for n in runnable if cur[n][0] == "yield"]
            if not busy and not self.delayed:
                if len(finished) == len(roles):
                    return
                idle_polls += 1
                if not polling or idle_polls > 8 * len(polling):
                    raise ProtocolError("deadlock: " + ", ".join("%s:%s" % (n, cur[n][:5] if cur[n] else None)
                                                                 for n in roles if n not in finished))
                cur[self.rng.choice(polling)] = None
                continue
            idle_polls = 0
            self.clock += 1
            ready = [i for i, (t, _) in enumerate(self.delayed) if t <= self.clock]
            if self.delayed and not busy and not ready:
                self.clock = min(t for t, _ in self.delayed)
                continue
            if ready and (not busy or self.rng.random() < 0.5):
                _, item = self.delayed.pop(self.rng.choice(ready))
                self._deliver(item)
                continue
            # some roles run slowly for a whole run, so that others get far ahead
            pool = [n for n in busy if n not in self.slow or self.rng.random() < 0.02] or busy
            pool = pool + [n for n in polling if self.rng.random() < 0.2]
            name = self.rng.choice(pool)
            op = cur[name]
            cur[name] = None
            if op[0] == "do":
                op[1]()

    @property
    def slow(self):
        if not hasattr(self, "_slow"):
            names = ["sp0", "sp1", "vp0", "vp1", "vp2", "sm0", "sm1", "s0", "s1", "s2", "s3", "pv", "epi",
                     "vmax", "recv", "fwd0", "fwd1", "sched0", "sched1"]
            self._slow = set(self.rng.sample(names, self.rng.randint(0, 3)))
        return self._slow


# planted mistakes, and the protocol form each applies to (None: both)
MUTATIONS = {"producers_uncoupled": None, "producers_skip_stage_free": None, "q_over_running_s": None, "q_waits_for_s_full": None, "epilogue_waits_for_pv_done": None,
             "sm_fin_without_wait": None, "two_fin_slots": None, "pv_over_unread_o": None,
             "scheduler_skips_free": None, "value_forwarder_skips_q": False,
             "issuers_uncoupled": False}


def run(sizes, seed, mutation=None, decoupled=True):
    Model(sizes, seed, mutation=mutation, decoupled=decoupled).run()
