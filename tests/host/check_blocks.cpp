// The order in which workgroups take the places of packed sequences: with
// rising starts every part of every sequence is some block's, once; with any
// starts a block's place and tokens stay inside the workspace and the tensors.
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <map>
#include <random>
#include <utility>
#include <vector>

#include "linear_places.h"

using namespace skinny;

#define CHECK(c, ...)                                                                                              \
    do {                                                                                                           \
        if (!(c)) {                                                                                                \
            fprintf(stderr, __VA_ARGS__);                                                                          \
            fprintf(stderr, "\n");                                                                                 \
            exit(1);                                                                                               \
        }                                                                                                          \
    } while (0)

// As the kernel does it: counts the sequences whose extra parts start by this one.
static bool locate(const std::vector<int> &starts, int tokens, int size, int block, int &place, Place &p)
{
    const int sequences = (int)starts.size() - 1;
    int seq = block;
    if (block >= sequences) {
        int count = 0;
        for (int i = 0; i < sequences; ++i)
            count += extra_starts_by(starts[i], tokens, size, block - sequences);
        if (count == 0)
            return false;
        seq = count - 1;
    }
    place = block_place(starts[seq], tokens, size, sequences, block, seq);
    return place_of(starts[seq], starts[seq + 1], tokens, size, place, seq, p);
}

int main()
{
    std::mt19937 rng(1);
    for (int round = 0; round < 20000; ++round) {
        const int sequences = 1 + (int)(rng() % 9), size = 64 * (1 + (int)(rng() % 4)), tokens = (int)(rng() % 2500);
        const int places = tokens / size + sequences;
        const bool rising = round % 3 != 2;
        std::vector<int> starts(sequences + 1);
        for (int &s : starts)
            s = rising ? (rng() % 4 ? (int)(rng() % (tokens + 1)) : (int)(rng() % (tokens / size + 1)) * size)
                       : (int)rng();
        if (rising) {
            starts[0] = 0;
            starts[sequences] = tokens;
            std::sort(starts.begin(), starts.end());
        }
        std::map<std::pair<int, int>, int> seen, used;
        for (int block = 0; block < places; ++block) {
            int place = -1;
            Place p;
            if (!locate(starts, tokens, size, block, place, p))
                continue;
            CHECK(place >= 0 && place < places, "round %d: block %d has place %d of %d", round, block, place, places);
            CHECK(p.first >= 0 && p.len >= 0 && p.first + p.len <= tokens, "round %d: tokens %d + %d of %d", round,
                  p.first, p.len, tokens);
            CHECK(p.part >= 0 && p.part < parts_of(p.len, size), "round %d: part %d", round, p.part);
            if (rising) {
                CHECK((!seen[{p.seq, p.part}]++), "round %d: part %d of sequence %d twice", round, p.part, p.seq);
                CHECK((!used[{place, 0}]++), "round %d: place %d twice", round, place);
                CHECK(place == first_place(starts[p.seq], tokens, size, p.seq) + p.part, "round %d: place %d", round,
                      place);
            }
        }
        if (rising)
            for (int i = 0; i < sequences; ++i)
                for (int j = 0; j < parts_of(starts[i + 1] - starts[i], size); ++j)
                    CHECK((seen[{i, j}]), "round %d: part %d of sequence %d is no block's", round, j, i);
    }
    puts("ok");
    return 0;
}
