// The block manager's reorder, unshare and truncate when the host's memory runs out
// at any of their allocations: a status, no exception across the C ABI, and nothing
// changed.  operator new counts down to a failure here; prints "ok" or what is wrong.
#include <cstdio>
#include <cstdlib>
#include <functional>
#include <new>
#include <vector>

#include "pa.h"

static long g_left = -1;   // allocations until one fails; negative: none does

void *operator new(std::size_t n) {
    if (g_left == 0) throw std::bad_alloc();
    if (g_left > 0) --g_left;
    if (void *p = std::malloc(n ? n : 1)) return p;
    throw std::bad_alloc();
}
void *operator new(std::size_t n, const std::nothrow_t &) noexcept { return std::malloc(n ? n : 1); }
void operator delete(void *p) noexcept { std::free(p); }
void operator delete(void *p, std::size_t) noexcept { std::free(p); }

namespace {

constexpr int kBlocks = 24, kSize = 4;

struct State {
    std::vector<int32_t> words;
    bool operator==(const State &o) const { return words == o.words; }
};

// Every table, length, count and total a caller can see.
State state_of(pa_bm *bm, const std::vector<int32_t> &seqs) {
    State s;
    for (int32_t q : seqs) {
        int32_t table[kBlocks], n = 0;
        int64_t tokens = 0;
        pa_bm_get_table(bm, q, table, kBlocks, &n, &tokens);
        s.words.insert(s.words.end(), table, table + kBlocks);
        s.words.push_back(n);
        s.words.push_back((int32_t)tokens);
    }
    for (int b = 0; b < kBlocks; ++b) s.words.push_back(pa_bm_refcount(bm, b));
    s.words.push_back((int32_t)pa_bm_num_free(bm));
    s.words.push_back((int32_t)pa_bm_num_cached(bm));
    s.words.push_back((int32_t)pa_bm_num_evictable(bm));
    return s;
}

// Four sequences whose blocks the prefix cache holds too (releasing them makes cache
// entries evictable), and chains of entries that only the cache holds (allocating
// evicts them).
pa_bm *make(std::vector<int32_t> &seqs) {
    pa_bm *bm = nullptr;
    pa_bm_create(&bm, kBlocks, kSize);
    std::vector<int32_t> tokens(64);
    for (int q = 0; q < 6; ++q) {
        int32_t id;
        int64_t inserted;
        pa_bm_add_seq(bm, &id);
        for (size_t i = 0; i < tokens.size(); ++i) tokens[i] = 1000 * q + (int)i;
        pa_bm_append_tokens(bm, id, 4 * kSize, nullptr, nullptr, nullptr);
        pa_bm_cache_seq(bm, id, tokens.data(), 4 * kSize, 7, &inserted);
        if (q < 4)
            seqs.push_back(id);
        else
            pa_bm_free_seq(bm, id);
    }
    return bm;
}

int run(const char *name, const std::function<pa_status(pa_bm *, const std::vector<int32_t> &)> &call) {
    for (long k = 0;; ++k) {
        std::vector<int32_t> seqs;
        pa_bm *bm = make(seqs);
        const State before = state_of(bm, seqs);
        pa_status st;
        g_left = k;
        try {
            st = call(bm, seqs);
        } catch (...) {
            g_left = -1;
            std::printf("%s: an exception left it at allocation %ld\n", name, k);
            return 1;
        }
        const bool failed = g_left == 0;
        g_left = -1;
        if (st != PA_OK && st != PA_ERR_NO_BLOCKS) {
            std::printf("%s: status %d at allocation %ld\n", name, (int)st, k);
            return 1;
        }
        if (st != PA_OK && !(state_of(bm, seqs) == before)) {
            std::printf("%s: changed, although it failed at allocation %ld\n", name, k);
            return 1;
        }
        // whatever happened, all blocks come back
        for (int32_t q : seqs) pa_bm_free_seq(bm, q);
        int64_t freed = 0;
        pa_bm_prefix_evict(bm, kBlocks, &freed);
        if (pa_bm_num_free(bm) != kBlocks) {
            std::printf("%s: %d of %d blocks free in the end, after allocation %ld\n", name, (int)pa_bm_num_free(bm),
                        kBlocks, k);
            return 1;
        }
        pa_bm_destroy(bm);
        if (st == PA_OK && !failed) return 0;
    }
}

}  // namespace

int main() {
    int bad = run("reorder", [](pa_bm *bm, const std::vector<int32_t> &s) {
        const int32_t parents[4] = {2, 2, 2, 2};
        return pa_bm_reorder(bm, s.data(), parents, 4);
    });
    bad += run("unshare", [](pa_bm *bm, const std::vector<int32_t> &s) {
        int32_t pairs[2 * kBlocks], n = 0;
        return pa_bm_unshare(bm, s[1], 0, pairs, kBlocks, &n);
    });
    bad += run("truncate", [](pa_bm *bm, const std::vector<int32_t> &s) { return pa_bm_truncate(bm, s[0], 3); });
    if (!bad) std::puts("ok");
    return bad;
}
