/* The argument checks of the page operators and of the attention over sequences
 * that begin alike, at the corners of splitzip_kv.h's limits: no call here gets
 * as far as a launch. */
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
    static const uint64_t corner[] = {0, 1, 7, 8, 63, 65, 255, 4095, 65535, 65536, 0x1000000, 0x7fffffff, 0x80000000u,
                                      0xfffffff8u, 0xffffffffu, 1ull << 40, (1ull << 63) - 8, (1ull << 63), ~7ull, ~0ull};
    const unsigned n = sizeof corner / sizeof *corner;
    uint16_t *k[1024], *v[1024];
    unsigned i, j;

    for (i = 0; i < 1024; ++i) {
        k[i] = (uint16_t *)(uintptr_t)(0x1000000ull * (i + 1));
        v[i] = (uint16_t *)(uintptr_t)(0x1000000ull * (i + 1) + 0x800000);
    }
    expect(splitzip_kv_pages_struct_size() == sizeof(splitzip_kv_pages) && splitzip_kv_groups_struct_size() == sizeof(splitzip_kv_groups),
           1, "sizes", 0);
    expect((int)splitzip_kv_pages_state_size(NULL), 0, "null cache", 0);
    expect((int)splitzip_kv_shared_workspace_size(NULL, 8, 1), 0, "null cache", 1);

    /* every pair of corners as shape: a size or 0 */
    for (i = 0; i < n; ++i)
        for (j = 0; j < n; ++j) {
            splitzip_kv_cache c = cache();
            c.batch = (uint32_t)corner[i];
            c.max_pages = (uint32_t)corner[j];
            expect(splitzip_kv_shared_workspace_size(&c, 64, 1) == splitzip_kv_shared_workspace_size(&c, 64, 65535), 1, "workspace",
                   i * n + j);
            c.num_pages = (uint32_t)corner[j];
            (void)splitzip_kv_pages_state_size(&c);
            c = cache();
            c.kv_heads = (uint32_t)corner[i];
            (void)splitzip_kv_shared_workspace_size(&c, (uint32_t)corner[j], (uint32_t)corner[i]);
            c.head_dim = (uint32_t)corner[j];
            c.page_size = (uint32_t)corner[i];
            (void)splitzip_kv_shared_workspace_size(&c, 8, 4);
        }

    /* strides out of reach, layers and states at the corners */
    for (i = 0; i < n; ++i)
        for (j = 0; j < 6; ++j) {
            splitzip_kv_cache c = cache(), good = cache();
            splitzip_kv_pages p = {0}, q = {0};
            if (corner[i] < 1ull << 40 && corner[i] % 8 == 0)
                continue;
            (j < 3 ? c.k_stride : c.v_stride)[j % 3] = corner[i];
            p.cache = &c;
            q.cache = &good;
            p.k = q.k = k;
            p.v = q.v = v;
            p.layers = q.layers = 1024;
            p.state = (void *)0x100000;
            p.state_bytes = SIZE_MAX;
            expect(splitzip_kv_pages_count(&p, NULL, NULL), SPLITZIP_ERR_INVALID, "count", i * 6 + j);
            expect(splitzip_kv_pages_resize(&p, (const int32_t *)0x5000, NULL, NULL), SPLITZIP_ERR_INVALID, "resize", i * 6 + j);
            expect(splitzip_kv_pages_copy(&p, &q, (const int32_t *)0x5000, (const int32_t *)0x5000, 1, NULL, NULL),
                   SPLITZIP_ERR_INVALID, "copy", i * 6 + j);
        }
    for (i = 0; i < n; ++i) {
        splitzip_kv_cache c = cache();
        splitzip_kv_pages p = {0};
        p.cache = &c;
        p.k = k;
        p.v = v;
        p.layers = (uint32_t)corner[i];
        p.state = (void *)0x100000;
        p.state_bytes = 0;
        expect(splitzip_kv_pages_fork(&p, (const int32_t *)0x5000, NULL, NULL),
               p.layers >= 1 && p.layers <= 1024 ? SPLITZIP_ERR_WORKSPACE : SPLITZIP_ERR_INVALID, "layers", i);
    }

    /* nulls, and the workspace that is too small */
    {
        splitzip_kv_cache c = cache();
        splitzip_kv_pages p = {0};
        splitzip_kv_query q = {0};
        splitzip_kv_groups g = {0};
        expect(splitzip_kv_pages_count(NULL, NULL, NULL), SPLITZIP_ERR_INVALID, "null pages", 0);
        expect(splitzip_kv_pages_fork(&p, NULL, NULL, NULL), SPLITZIP_ERR_INVALID, "no cache", 0);
        expect(splitzip_kv_pages_compact(&p, NULL, NULL, NULL, NULL), SPLITZIP_ERR_INVALID, "no cache", 1);
        expect(splitzip_kv_pages_copy(&p, NULL, NULL, NULL, 0, NULL, NULL), SPLITZIP_ERR_INVALID, "null pages", 1);
        p.cache = &c;
        expect(splitzip_kv_pages_resize(&p, NULL, NULL, NULL), SPLITZIP_ERR_INVALID, "no pools", 0);
        expect(splitzip_kv_attend_shared(NULL, &q, &g, NULL, 0, NULL, NULL), SPLITZIP_ERR_INVALID, "null cache", 2);
        expect(splitzip_kv_attend_shared(&c, NULL, &g, NULL, 0, NULL, NULL), SPLITZIP_ERR_INVALID, "null query", 0);
        expect(splitzip_kv_attend_shared(&c, &q, NULL, NULL, 0, NULL, NULL), SPLITZIP_ERR_INVALID, "null groups", 0);
        q.q = (const uint16_t *)0x30000;
        q.out = (uint16_t *)0x40000;
        q.heads = 16;
        q.window = SPLITZIP_KV_ALL;
        expect(splitzip_kv_attend_shared(&c, &q, &g, (void *)0x50000, 0, NULL, NULL), SPLITZIP_ERR_WORKSPACE, "no workspace", 0);
        for (i = 0; i < n; ++i) {
            g.groups = (uint32_t)corner[i];
            expect(splitzip_kv_attend_shared(&c, &q, &g, (void *)0x50000, 0, NULL, NULL),
                   g.groups ? SPLITZIP_ERR_INVALID : SPLITZIP_ERR_WORKSPACE, "groups", i);
        }
    }
    printf("%d failures\n", failures);
    return failures ? EXIT_FAILURE : EXIT_SUCCESS;
}
