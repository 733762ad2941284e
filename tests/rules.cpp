// Prints what the library's rules say on 256 CUs: a line "own T WORKGROUPS" of its input asks
// whether the experts' workgroups choose for themselves.
#include <cstdint>
#include <cstdio>
#include <cstring>

namespace convrot {
bool moe_own_choice(int T, int64_t workgroups, int64_t cus);
} // namespace convrot

int main()
{
    char rule[16];
    long long a, b;
    while (std::scanf("%15s %lld %lld", rule, &a, &b) == 3)
        if (!std::strcmp(rule, "own")) std::printf("%d\n", convrot::moe_own_choice((int)a, b, 256));
        else return 1;
}
