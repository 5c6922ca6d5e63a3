/*
 * Driver for the sanitizer run of the paged K/V calls' host code (TEST
 * INFRASTRUCTURE): linked with api_kv.hip and api.hip built with host-side
 * ASan/UBSan by tests/test_sanitizers.py, on a machine without a GPU.  Each
 * struct field and argument takes values at the ends of its range in turn and at random; every
 * call has to come back with a status and, where it refuses, a message.
 * Never dereferences the fake addresses it passes.
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "ibp_kv.h"

static uint64_t state = 88172645463325252ull;
static uint64_t rnd(void)
{
    state ^= state << 13;
    state ^= state >> 7;
    state ^= state << 17;
    return state;
}

static const uint64_t ends[] = {0, 1, 2, 3, 7, 8, 16, 64, 128, 256, 264, 1024, 4096, 4097, 65535, 65536, 65537,
                                1u << 20, 1u << 24, 1u << 30, (1u << 30) + 1, 0x7FFFFFFFu, 0x80000000u,
                                0xFFFFFFFFu, 1ull << 32, 1ull << 40, 1ull << 62, 1ull << 63, ~0ull, ~7ull};
/* mostly `usual`, else one of the ends */
static uint64_t pick(uint64_t usual) { return rnd() % 12 ? usual : ends[rnd() % (sizeof ends / sizeof *ends)]; }
static void *address(uint64_t usual) { return (void *)(uintptr_t)pick(usual << 20); }

static long calls, refusals, no_device;
static void came_back(int status, const char *what)
{
    const char *msg = ibp_last_error();
    ++calls;
    if (status == IBP_ERR_HIP) ++no_device;
    else if (status < 0) ++refusals;
    if (status < 0 && (!msg || !msg[0])) printf("%s: status %d without a message\n", what, status);
    if (status > 0) printf("%s: status %d\n", what, status);
}

static ibp_kv_rows rows(uint64_t at, uint32_t heads)
{
    ibp_kv_rows r;
    r.data = address(at);
    r.token_stride = pick(64 * heads);
    r.head_stride = pick(64);
    r.n_heads = (uint32_t)pick(heads);
    return r;
}

int main(void)
{
    for (int i = 0; i < 200000; ++i) {
        ibp_kv_cache c;
        c.k = address(1);
        c.v = address(2);
        c.n_pages = pick(10);
        c.n_heads = (uint32_t)pick(2);
        c.head_dim = (uint32_t)pick(64);
        c.page_tokens = (uint32_t)pick(16);
        c.dtype = (uint32_t)(rnd() % 20 ? rnd() % 2 : pick(2));
        c.head_stride = pick(64);
        c.token_stride = pick(128);
        c.page_stride = pick(2048);
        ibp_kv_batch b;
        b.q_start = address(3);
        b.kv_len = address(4);
        b.page_table = address(5);
        b.table_stride = pick(8);
        b.n_rows = pick(3);
        b.n_seqs = (uint32_t)pick(3);
        b.max_q = (uint32_t)pick(4);
        b.max_kv = (uint32_t)pick(128);
        ibp_kv_rows k = rows(6, 2), v = rows(7, 2), q = rows(8, 4), o = rows(9, 4);
        if (rnd() % 4 == 0) {  /* near each other, the same strides: looked at for overlaps */
            o = q;
            o.data = (void *)((uintptr_t)q.data + 16 * (rnd() % 64) - 16 * (rnd() % 64));
        }
        const uint32_t n = (uint32_t)pick(8);
        const float scale = (float)(rnd() % 9 ? 0.125 : rnd() % 2 ? INFINITY : NAN);
        uint64_t bytes = 0;
        const ibp_kv_cache *pc = rnd() % 50 ? &c : NULL;
        const ibp_kv_batch *pb = rnd() % 50 ? &b : NULL;
        const ibp_kv_rows *pq = rnd() % 50 ? &q : NULL;
        came_back(ibp_kv_append(pc, &k, &v, pq, rnd() % 50 ? &o : NULL, address(10), address(11), pick(3),
                                address(12), pick(9), (uint32_t)pick(64), address(13), address(14), scale,
                                (unsigned)(rnd() % 3), NULL), "append");
        came_back(ibp_kv_page_bounds(pc, pb, address(15), NULL), "page_bounds");
        came_back(ibp_kv_attend(pc, pb, pq, &o, scale, (uint32_t)pick(0), (unsigned)(rnd() % 3), address(16),
                                address(17), pick(1 << 20), NULL), "attend");
        came_back(ibp_kv_attend_workspace(pc, pb, (uint32_t)pick(4), rnd() % 50 ? &bytes : NULL),
                  "attend_workspace");
        came_back(ibp_kv_select(pc, pb, address(18), pick(10), pq, (uint32_t)pick(1), (uint32_t)pick(1), n,
                                address(19), address(20), pick(1 << 20), NULL), "select");
        came_back(ibp_kv_select_workspace(pc, pb, n, rnd() % 50 ? &bytes : NULL), "select_workspace");
        came_back(ibp_kv_attend_selected(pc, pb, pq, &o, address(21), n, scale, address(22), address(23),
                                         pick(1 << 20), NULL), "attend_selected");
        came_back(ibp_kv_attend_selected_workspace(pc, pb, (uint32_t)pick(4), n, rnd() % 50 ? &bytes : NULL),
                  "attend_selected_workspace");
    }
    printf("%ld calls, %ld refused, %ld without a device\n", calls, refusals, no_device);
    if (refusals > calls / 10 && no_device > calls / 50) printf("kv sanitizer run ok\n");
    return 0;
}
