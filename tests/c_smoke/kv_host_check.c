/* The argument checks of splitzip_kv.h at the corners of its limits: no call
 * here gets as far as a launch. */
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "splitzip_kv.h"

static int failures;

static void expect(int got, int want, const char *what, unsigned long long i)
{
    if (got != want) {
        printf("%s, case %llu: %d instead of %d\n", what, i, got, want);
        ++failures;
    }
}

static splitzip_kv_cache cache(void)
{
    splitzip_kv_cache c = {0};
    c.k = (uint16_t *)0x10000;
    c.v = (uint16_t *)0x20000;
    c.k_stride[0] = c.v_stride[0] = 8 * 16 * 64;
    c.k_stride[1] = c.v_stride[1] = 16 * 64;
    c.k_stride[2] = c.v_stride[2] = 64;
    c.table = (const int32_t *)0x3000;
    c.table_stride = 4;
    c.lens = (int32_t *)0x4000;
    c.num_pages = 10;
    c.page_size = 16;
    c.kv_heads = 8;
    c.head_dim = 64;
    c.batch = 2;
    c.max_pages = 4;
    return c;
}

int main(void)
{
    static const uint64_t corner[] = {0, 1, 7, 8, 63, 65, 255, 4095, 65535, 65536, 0x7fffffff, 0x80000000u, 0xfffffff8u,
                                      0xffffffffu, 1ull << 40, (1ull << 63) - 8, (1ull << 63), ~7ull, ~0ull};
    const unsigned n = sizeof corner / sizeof *corner;
    size_t sizes[4];
    unsigned i, j;

    splitzip_kv_struct_sizes(sizes);
    expect(sizes[0] == sizeof(splitzip_kv_cache) && sizes[1] == sizeof(splitzip_kv_rows) &&
               sizes[2] == sizeof(splitzip_kv_query) && sizes[3] == sizeof(splitzip_kv_budget), 1, "sizes", 0);

    /* every pair of corners as shape: a size or 0, and more mass never less */
    for (i = 0; i < n; ++i)
        for (j = 0; j < n; ++j) {
            splitzip_kv_cache c = cache();
            size_t a, b;
            c.batch = (uint32_t)corner[i];
            c.max_pages = (uint32_t)corner[j];
            a = splitzip_kv_attend_workspace_size(&c, 64, 0);
            b = splitzip_kv_attend_workspace_size(&c, 64, 0xffffffffu);
            expect(b == 0 || b >= a, 1, "workspace", i * n + j);
            c = cache();
            c.kv_heads = (uint32_t)corner[i];
            (void)splitzip_kv_attend_workspace_size(&c, (uint32_t)corner[j], (uint32_t)corner[i]);
            c.head_dim = (uint32_t)corner[j];
            c.page_size = (uint32_t)corner[i];
            (void)splitzip_kv_attend_workspace_size(&c, 8, 64);
        }

    /* strides out of reach, one at a time */
    for (i = 0; i < n; ++i)
        for (j = 0; j < 6; ++j) {
            splitzip_kv_cache c = cache();
            splitzip_kv_rows r = {0};
            if (corner[i] < 1ull << 40 && corner[i] % 8 == 0)
                continue;
            (j < 3 ? c.k_stride : c.v_stride)[j % 3] = corner[i];
            expect(splitzip_kv_append(&c, &r, NULL, NULL), SPLITZIP_ERR_INVALID, "append", i * 6 + j);
            expect(splitzip_kv_gather(&c, &r, NULL, NULL), SPLITZIP_ERR_INVALID, "gather", i * 6 + j);
        }
    for (i = 0; i < n; ++i)
        for (j = 0; j < 4; ++j) {
            splitzip_kv_cache c = cache();
            splitzip_kv_rows r = {0};
            if (corner[i] < 1ull << 40 && corner[i] % 8 == 0)
                continue;
            r.rows = 5;
            (j < 2 ? r.k_stride : r.v_stride)[j % 2] = corner[i];
            expect(splitzip_kv_append(&c, &r, NULL, NULL), SPLITZIP_ERR_INVALID, "rows", i * 4 + j);
        }

    /* nulls, and a budget at every corner without the mass */
    {
        splitzip_kv_cache c = cache();
        splitzip_kv_rows r = {0};
        splitzip_kv_query q = {0};
        splitzip_kv_budget b = {0};
        expect(splitzip_kv_append(NULL, &r, NULL, NULL), SPLITZIP_ERR_INVALID, "null cache", 0);
        expect(splitzip_kv_append(&c, NULL, NULL, NULL), SPLITZIP_ERR_INVALID, "null rows", 0);
        expect(splitzip_kv_gather(&c, NULL, NULL, NULL), SPLITZIP_ERR_INVALID, "null rows", 1);
        expect(splitzip_kv_append(&c, &r, NULL, NULL), SPLITZIP_OK, "no rows", 0);
        expect(splitzip_kv_attend(NULL, &q, NULL, 0, NULL, NULL), SPLITZIP_ERR_INVALID, "null cache", 1);
        expect(splitzip_kv_attend(&c, NULL, NULL, 0, NULL, NULL), SPLITZIP_ERR_INVALID, "null query", 0);
        expect(splitzip_kv_attend(&c, &q, NULL, 0, NULL, NULL), SPLITZIP_ERR_INVALID, "zero query", 0);
        expect(splitzip_kv_evict(&c, NULL, &b, NULL, NULL), SPLITZIP_ERR_INVALID, "null destination", 0);
        expect(splitzip_kv_evict(&c, &c, NULL, NULL, NULL), SPLITZIP_ERR_INVALID, "null budget", 0);
        expect((int)splitzip_kv_attend_workspace_size(NULL, 8, 0), 0, "null cache", 2);
        q.q = (const uint16_t *)0x30000;
        q.out = (uint16_t *)0x40000;
        q.heads = 16;
        expect(splitzip_kv_attend(&c, &q, (void *)0x50000, 0, NULL, NULL), SPLITZIP_ERR_WORKSPACE, "no workspace", 0);
        for (i = 0; i < n; ++i)
            for (j = 0; j < n; ++j) {
                b.budget = (uint32_t)corner[i];
                b.sinks = b.recent = (uint32_t)corner[j];
                expect(splitzip_kv_evict(&c, &c, &b, NULL, NULL), SPLITZIP_ERR_INVALID, "budget", i * n + j);
            }
    }
    printf("%d failures\n", failures);
    return failures ? EXIT_FAILURE : EXIT_SUCCESS;
}
