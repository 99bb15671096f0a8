// Test shim: the signals between the warps of the distillation gradient's
// pipeline (distill.cu) for one CTA, explored state by state on the host with the
// slices and mbarriers of grad_signals.cuh.
//
// A state is how far every warp (or group of workers) has come, which rows'
// copies have begun and which are there, and whether a wait was given up.  From
// each state every warp that can go on takes its next step, and every copy in
// flight may arrive.
#include <cstdio>
#include <unordered_set>
#include <vector>

#include "grad_signals.cuh"

namespace {

enum Kind { kArrive, kWait, kFullWait, kUse, kLook, kCopy, kDrain };
enum Bar { kReady, kEntries, kSums, kScalars, kStored, kPassed, kBars };
const char* const kNames[] = {"ready", "entries", "sums", "scalars", "stored", "passed"};
constexpr int kWarps = 9, kMaxRows = 8;

struct Step {
    int kind, bar, n;
};
struct Place {
    int warp, step;
};
struct State {
    uint8_t at[kWarps] = {};
    uint8_t begun = 0, there = 0;  // bits: rows
    uint8_t given_up = 0, off = 0;  // a wait was given up; warp D has seen it
    bool operator==(const State& o) const {
        for (int i = 0; i < kWarps; ++i)
            if (at[i] != o.at[i]) return false;
        return begun == o.begun && there == o.there && given_up == o.given_up && off == o.off;
    }
};
struct Hash {
    size_t operator()(const State& s) const {
        uint64_t h = s.begun | uint64_t(s.there) << 8 | uint64_t(s.given_up) << 16 | uint64_t(s.off) << 17;
        for (int i = 0; i < kWarps; ++i) h = (h ^ s.at[i]) * 0x9E3779B97F4A7C15ull, h ^= h >> 29;
        return h;
    }
};

struct Explorer {
    int rows, barriers;  // mbarriers of copies: the library's kFull, or fewer to see what that does
    unsigned masked;
    bool may_give_up;
    bool hasty;  // warps A no longer wait for passed once a wait was given up
    char* fault;
    int fault_size;
    std::vector<Step> prog[kWarps];
    std::vector<Place> parties[kBars][kMaxRows];
    std::unordered_set<State, Hash> seen;
    std::vector<State> todo;
    bool failed = false;

    int full(int n) const { return barriers == dspark::kFull ? dspark::full_of(n) : n % barriers; }
    unsigned parity(int n) const { return barriers == dspark::kFull ? dspark::full_parity(n) : n / barriers & 1; }

    void fail(const char* what, const char* name, int n) {
        if (!failed) snprintf(fault, fault_size, "%s %s(%d)", what, name, n);
        failed = true;
    }
    void sync(int warp, int bar, int n) {
        prog[warp].push_back({kArrive, bar, n});
        prog[warp].push_back({kWait, bar, n});
    }
    void arrive(int warp, int bar, int n) { prog[warp].push_back({kArrive, bar, n}); }

    // The warps' steps, in the kernel's order.
    void programs() {
        for (int own = 0; own < 2; ++own)
            for (int n = own; n < rows; n += 2) {
                const int A = own, W = 2 + own, B = 4 + own, C = 6 + own;
                if (n > 1) sync(A, kPassed, n - 2);
                prog[A].push_back({kFullWait, 0, n});
                prog[A].push_back({kUse, 0, n});
                arrive(A, kReady, n);
                arrive(A, kEntries, n);
                sync(W, kReady, n);
                prog[W].push_back({kUse, 0, n});
                arrive(W, kSums, n);
                sync(W, kScalars, n);
                prog[W].push_back({kUse, 0, n});
                arrive(W, kStored, n);
                sync(B, kEntries, n);
                sync(B, kSums, n);
                arrive(B, kScalars, n);
                sync(C, kScalars, n);
                if (n + 2 < rows) arrive(C, kPassed, n);
                sync(C, kStored, n);
            }
        auto copy = [&](int n) {
            if (n >= rows) return;
            prog[8].push_back({kLook, 0, n});
            prog[8].push_back({kCopy, 0, n});
        };
        for (int n = 0; n < dspark::kSlices; ++n) copy(n);
        for (int n = 0; n < rows; ++n) {
            sync(8, kStored, n);
            copy(n + dspark::kSlices);
        }
        prog[8].push_back({kDrain, 0, 0});
        for (int i = 0; i < kWarps; ++i)
            for (int k = 0; k < static_cast<int>(prog[i].size()); ++k)
                if (prog[i][k].kind == kArrive) parties[prog[i][k].bar][prog[i][k].n].push_back({i, k});
    }

    bool complete(const State& s, int bar, int n) const {
        for (const Place& q : parties[bar][n])
            if (s.at[q.warp] <= q.step) return false;
        return true;
    }
    // Whether a wait for row n's copy returns: the phase in progress has another parity.
    bool returns(const State& s, int n) const {
        unsigned phases = 0;
        for (int m = 0; m < rows; ++m) phases += full(m) == full(n) && (s.there >> m & 1);
        return (phases & 1) != parity(n);
    }
    // A wait that is over changes nothing for the others: it is passed at once.
    void add(State s) {
        for (bool moved = true; moved;) {
            moved = false;
            for (int i = 0; i < kWarps; ++i)
                if (s.at[i] < prog[i].size()) {
                    const Step& t = prog[i][s.at[i]];
                    if (t.kind == kWait && (complete(s, t.bar, t.n) || (hasty && s.given_up && t.bar == kPassed)))
                        ++s.at[i], moved = true;
                }
        }
        if (seen.insert(s).second) todo.push_back(s);
    }

    void step(const State& s) {
        const unsigned flying = s.begun & ~s.there;
        bool any = false, ended = true;
        auto go = [&](const State& to) {
            any = true;
            add(to);
        };
        for (int n = 0; n < rows; ++n)
            if (flying >> n & 1) {
                State to = s;
                to.there |= 1u << n;
                go(to);
            }
        if (may_give_up && !s.given_up) {  // a wait for another CTA's sums or losses
            State to = s;
            to.given_up = 1;
            go(to);
        }
        for (int i = 0; i < kWarps; ++i) {
            if (s.at[i] == prog[i].size()) continue;
            ended = false;
            const Step& t = prog[i][s.at[i]];
            const int n = t.n;
            State to = s;
            ++to.at[i];
            switch (t.kind) {
                case kArrive:
                    if (n >= 2 && !complete(s, t.bar, n - 2)) return fail("signalled before the row before the last:", kNames[t.bar], n);
                    break;
                case kWait:
                    continue;
                case kFullWait:
                    if (!s.given_up && !returns(s, n)) {
                        if (!may_give_up) continue;
                        to.given_up = 1;
                    }
                    break;
                case kUse:
                    if (s.given_up) break;  // the row is void
                    if (!(s.begun >> n & 1)) return fail("taken before its copy is issued:", "slice of row", n);
                    for (int m = 0; m < rows; ++m)
                        if (dspark::slice_of(m) == dspark::slice_of(n)) {
                            if (m > n && (s.begun >> m & 1)) return fail("taken after the next copy is issued:", "slice of row", n);
                            if (flying >> m & 1) return fail("taken while a copy lands in it:", "slice of row", n);
                        }
                    break;
                case kLook:
                    to.off |= s.given_up;
                    break;
                case kCopy:
                    if (s.off) break;
                    for (int m = 0; m < rows; ++m)
                        if (flying >> m & 1) {
                            if (full(m) == full(n)) return fail("arrival in a phase in progress:", "row", n);
                            if (dspark::slice_of(m) == dspark::slice_of(n)) return fail("begins where another lands:", "copy", n);
                        }
                    to.begun |= 1u << n;
                    if (masked >> n & 1) to.there |= 1u << n;  // an arrival alone
                    break;
                case kDrain:
                    if (s.given_up) {
                        bool over = true;
                        int begun = 0;
                        while (s.begun >> begun) ++begun;
                        for (int m = begun > dspark::kFull ? begun - dspark::kFull : 0; m < begun; ++m) over = over && returns(s, m);
                        if (!over) continue;
                    }
                    break;
            }
            go(to);
        }
        if (ended && flying) return fail("in flight at the end:", "a copy of", static_cast<int>(flying));
        if (!ended && !any) fail("no warp can go on:", "row", 0);
    }
};

}  // namespace

// The number of states reached, or -1 with the fault found.
extern "C" long long grad_explore(int rows, unsigned masked, int barriers, int may_give_up, int hasty, char* fault,
                                  int fault_size) {
    if (rows < 1 || rows > kMaxRows || barriers < 1) return -2;
    Explorer e;
    e.rows = rows;
    e.barriers = barriers;
    e.masked = masked;
    e.may_give_up = may_give_up != 0;
    e.hasty = hasty != 0;
    e.fault = fault;
    e.fault_size = fault_size;
    e.programs();
    e.add(State{});
    while (!e.todo.empty() && !e.failed) {
        const State s = e.todo.back();
        e.todo.pop_back();
        e.step(s);
    }
    return e.failed ? -1 : static_cast<long long>(e.seen.size());
}
extern "C" int grad_barriers() { return dspark::kFull; }
