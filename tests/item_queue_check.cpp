// Walks every interleaving of the item queue (item_queue.cuh): a publisher, two markers and two readers over a few
// items, each step of each an event of its own. A marker that holds a marked item writes the mark; a reader that holds an
// item reads its place at any time before it takes the next one. Prints the number of states, and the number of reads
// that saw something else than whether their item is marked, for the header's rule and for a rule that clears the
// place of four items ago instead (which must be seen to fail). The second marker is held to what the V stages
// allow it, one item ahead of the first: it cannot pass an item that the first has not been through.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <set>
#include <vector>

#include "item_queue.cuh"

using namespace duo;

constexpr int kItems = 14;

struct State {
    signed char published;  // items published
    signed char taken[4];   // items taken by markers 0, 1 and readers 2, 3; the last one taken is held
    signed char done[4];    // 1: the marker has written (or skipped) its mark, the reader has read
    signed char place[kItemMarks];
    bool operator<(const State& o) const { return std::memcmp(this, &o, sizeof(State)) < 0; }
};

static long wrong;
static unsigned pattern;  // bit i: item i is marked
static bool clears;       // the other rule

static bool marked(int i) { return (pattern >> i) & 1u; }

static void push(std::vector<State>& todo, std::set<State>& seen, const State& s) {
    if (seen.insert(s).second) todo.push_back(s);
}

static size_t walk() {
    State s;
    std::memset(&s, 0, sizeof(s));
    std::memset(s.place, clears ? 0 : kNoItem, sizeof(s.place));
    for (signed char& d : s.done) d = 1;
    std::set<State> seen;
    std::vector<State> todo;
    push(todo, seen, s);
    while (!todo.empty()) {
        s = todo.back();
        todo.pop_back();
        bool room = s.published < kItems;
        if (s.published >= kQueueSlots)
            for (int c = 0; c < 4; ++c) room = room && s.taken[c] > s.published - kQueueSlots;
        if (room) {
            State n = s;
            ++n.published;
            push(todo, seen, n);
        }
        for (int c = 0; c < 4; ++c) {
            const int held = s.taken[c] - 1;
            if (s.done[c] && s.taken[c] < s.published && !(c == 1 && s.taken[1] > s.taken[0])) {
                State n = s;
                ++n.taken[c];
                n.done[c] = 0;
                if (clears && c == 0) n.place[(held + 1 + 4) % 8] = 0;
                push(todo, seen, n);
            }
            if (!s.done[c]) {
                State n = s;
                n.done[c] = 1;
                if (c < 2) {
                    if (marked(held)) n.place[mark_place(held)] = clears ? 1 : held;
                    push(todo, seen, n);
                } else if (s.taken[0] > held && s.taken[1] > held && (s.taken[0] > held + 1 || s.done[0]) &&
                           (s.taken[1] > held + 1 || s.done[1])) {  // reads behind both markers' look at the item
                    const bool got = clears ? s.place[mark_place(held)] != 0 : s.place[mark_place(held)] == held;
                    if (got != marked(held)) ++wrong;
                    push(todo, seen, n);
                }
            }
        }
    }
    return seen.size();
}

int main() {
    const unsigned patterns[] = {0x0000u, 0x3FFFu, 0x0001u, 0x0101u, 0x1555u, 0x2AAAu, 0x00F0u};
    for (int rule = 0; rule < 2; ++rule) {
        clears = rule == 1;
        wrong = 0;
        size_t states = 0;
        for (unsigned p : patterns) {
            pattern = p;
            states += walk();
        }
        std::printf("%s %zu %ld\n", clears ? "clears" : "marks", states, wrong);
    }
    return 0;
}
