// pkv_bm_evict_batch when host memory runs out: every allocation that the call makes is failed in turn,
// and the manager must be as it was before (tests/test_block_manager_memory.py builds and runs this).
#include <cstdio>
#include <cstdlib>
#include <new>

#include "block_manager.cpp"

static long countdown = -1;  // the allocation to fail, counted from 0; < 0: none
void* operator new(size_t n) {
    if (countdown >= 0 && countdown-- == 0) throw std::bad_alloc();
    void* p = malloc(n ? n : 1);
    if (!p) throw std::bad_alloc();
    return p;
}
void operator delete(void* p) noexcept { free(p); }
void operator delete(void* p, size_t) noexcept { free(p); }

namespace pkv {
pkv_status fail(pkv_status st, const char*, ...) { return st; }
}  // namespace pkv

#define CHECK(x)                                            \
    do {                                                    \
        if (!(x)) {                                         \
            printf("line %d (after %ld): %s\n", __LINE__, k, #x); \
            return 1;                                       \
        }                                                   \
    } while (0)

int main() {
    constexpr int kSeqs = 3, kTokens = 16 * 700, kBudget = 16 * 3 + 5, kNew = 4;
    std::vector<int32_t> toks(kTokens);
    for (int i = 0; i < kTokens; ++i) toks[i] = i;
    for (int cache = 0; cache < 2; ++cache) {
        long failed = 0;
        for (long k = 0;; ++k) {
            pkv_block_manager* bm = nullptr;
            CHECK(pkv_bm_create(4000, 16, nullptr, cache, &bm) == PKV_OK);
            int64_t ids[kSeqs], cached;
            for (int s = 0; s < kSeqs; ++s) {
                toks[0] = -s;  // nothing in common
                CHECK(pkv_bm_add_sequence(bm, toks.data(), kTokens - s, nullptr, 0, ids + s, &cached) == PKV_OK);
            }
            std::vector<int32_t> before(kSeqs * 700), after(kSeqs * 700), lens(kSeqs), tab(kSeqs * kNew), nl(kSeqs);
            pkv_bm_stats s0, s1;
            CHECK(pkv_bm_batch_tables(bm, ids, kSeqs, before.data(), 700, lens.data()) == PKV_OK);
            CHECK(pkv_bm_get_stats(bm, &s0) == PKV_OK);
            countdown = k;
            const pkv_status st = pkv_bm_evict_batch(bm, ids, kSeqs, kBudget, tab.data(), kNew, nl.data());
            const bool reached = countdown < 0;  // an allocation failed
            countdown = -1;
            if (reached) {
                ++failed;
                CHECK(st != PKV_OK);
                CHECK(pkv_bm_batch_tables(bm, ids, kSeqs, after.data(), 700, nl.data()) == PKV_OK);
                CHECK(after == before && nl == lens);
                CHECK(pkv_bm_get_stats(bm, &s1) == PKV_OK);
                CHECK(memcmp(&s0, &s1, sizeof s0) == 0);
            } else {
                CHECK(st == PKV_OK && nl[0] == kBudget);
                CHECK(pkv_bm_get_stats(bm, &s1) == PKV_OK);
                CHECK(s1.used_blocks == kSeqs * kNew);
                CHECK(s1.free_blocks + s1.parked_blocks + s1.used_blocks == 4000);
            }
            pkv_bm_destroy(bm);
            if (!reached) break;
        }
        printf("prefix cache %d: %ld allocations failed in turn\n", cache, failed);
        if (failed < 5) return 1;
    }
    return 0;
}
